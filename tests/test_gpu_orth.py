"""Newton-Schulz orthogonalisation and the Muon update on the GPU against the
float64 oracle.

Tolerance. One step maps singular values by p(t) = a t + b t^3 + c t^5, whose
slope is at most 4 on [0, 1.21], so a rounding error made at step i reaches
the result at most 4^(5 - i) times. The matrix entering step i has a Frobenius
norm of at most 3.4445^i (X_0 has 1); a step stores and multiplies it with
relative errors of 2^-22 (two fp16 parts), at most six of them. So
  ||E||_F <= sum_i 4^(5 - i) 3.4445^i 6 2^-22 <= 5 4^5 6 2^-22 = 7.3e-3
whatever the size, far above what is seen, and below one wrong entry of any
tested matrix (entries are about 1 / sqrt(longer side)). A bf16 result may be
off by half a unit (2^-8 of the value) on top of it, entry by entry.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from oracle import norm_update_oracle as ou

pytestmark = pytest.mark.gpu
TOL = 7.3e-3
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


def _np(t):
    return t.detach().double().cpu().numpy()


def _randn(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed))


def _ws(n, rows, cols, steps=5):
    return moe.workspace(moe.moe_orthogonalize_workspace_size(n, rows, cols, steps))


def _orth(g, out_dtype=F32, steps=5, eps=1e-7):
    n, rows, cols = g.shape
    out = torch.full(g.shape, 7.0, dtype=out_dtype, device="cuda")
    # a workspace full of NaN: nothing in it is read before it is written
    moe.moe_orthogonalize(g, out, _ws(n, rows, cols, steps).fill_(0xFF), steps=steps, eps=eps)
    torch.cuda.synchronize()
    return out


def _excess(got, ref, half):
    """Frobenius norm of what exceeds the output's own rounding."""
    assert np.isfinite(got).all()
    return np.linalg.norm(np.maximum(np.abs(got - ref) - half * np.abs(ref), 0.0))


SHAPES = [(1, 1, 1), (2, 1, 70), (2, 70, 1), (2, 5, 3), (1, 31, 33), (2, 32, 32), (3, 64, 200),
          (2, 129, 127), (1, 257, 300), (1, 128, 513), (2, 300, 96), (1, 640, 384),
          (5, 33, 1100), (1, 1000, 130)]


@pytest.mark.parametrize("g_dtype,out_dtype", [(F32, F32), (F32, BF16), (BF16, BF16),
                                               (BF16, F32)])
@pytest.mark.parametrize("n,rows,cols", SHAPES)
def test_orthogonalize(n, rows, cols, g_dtype, out_dtype):
    print(f"[orth] n={n} {rows}x{cols} {g_dtype} -> {out_dtype}", flush=True)
    g = (_randn(n, rows, cols, seed=rows + cols) * 1e-3).to(g_dtype).cuda()
    out = _np(_orth(g, out_dtype))
    for i in range(n):
        assert _excess(out[i], ou.orthogonalize(_np(g[i])), HALF[out_dtype]) <= TOL, i


# Batches whose products take 128 x 128 tiles (300 and more of them) and
# 256 x 256 ones (252 of sides that end inside a tile), wide, tall and square;
# the first, a middle and the last matrix are compared, and that no other row
# is left unwritten.
MANY = [(50, 301, 333), (50, 333, 301), (42, 750, 801), (42, 801, 750), (42, 768, 768)]


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("n,rows,cols", MANY)
def test_many_matrices(n, rows, cols, out_dtype):
    print(f"[orth] n={n} {rows}x{cols} {out_dtype}", flush=True)
    g = torch.randn(n, rows, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(n))
    out = _orth(g, out_dtype)
    assert torch.isfinite(out).all() and float(out.abs().max()) < 1.3
    for i in (0, n // 2, n - 1):
        assert _excess(_np(out[i]), ou.orthogonalize(_np(g[i])), HALF[out_dtype]) <= TOL, i


# Short sides of one to four 32-row blocks: the next step's Gram product from
# one workgroup of a matrix, from several of which the last has fewer blocks, or
# from a launch of its own (long sides; many matrices).
SHORT = [(300, 20, 60), (2, 2000, 30), (1, 17, 5000), (300, 100, 64), (2, 50, 700), (90, 64, 500),
         (2, 90, 380), (2, 300, 90), (3, 120, 300), (2, 270, 128), (40, 128, 520)]


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("n,rows,cols", SHORT)
def test_short_sides(n, rows, cols, out_dtype):
    print(f"[orth] n={n} {rows}x{cols} {out_dtype}", flush=True)
    g = _randn(n, rows, cols, seed=n + cols).cuda()
    out = _orth(g, out_dtype)
    assert torch.isfinite(out).all() and float(out.abs().max()) < 1.3
    assert torch.equal(out, _orth(g, out_dtype))
    for i in (0, n // 2, n - 1):
        assert _excess(_np(out[i]), ou.orthogonalize(_np(g[i])), HALF[out_dtype]) <= TOL, i


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("rows,cols", [(96, 160), (200, 70)])
def test_steps(rows, cols, steps):
    print(f"[orth] steps={steps} {rows}x{cols}", flush=True)
    g = _randn(2, rows, cols, seed=steps).cuda()
    out = _np(_orth(g, steps=steps))
    # the bound's sum for this many steps
    tol = max(TOL, steps * 4.0 ** steps * 6 * 2.0 ** -22)
    for i in range(2):
        assert _excess(out[i], ou.orthogonalize(_np(g[i]), steps), 2 * U) <= tol


@pytest.mark.parametrize("rank", [1, 2, 8])
def test_low_rank(rank):
    """Gradients of experts with few tokens: all other directions are noise
    that the iteration amplifies."""
    a, b = _randn(200, rank, seed=1), _randn(rank, 330, seed=2)
    g = torch.stack([a @ b, (a @ b) * 1e-4]).cuda()
    out = _np(_orth(g))
    for i in range(2):
        assert _excess(out[i], ou.orthogonalize(_np(g[i])), U) <= TOL


def test_scales_of_gradients():
    """Squares of the largest and smallest would leave fp32's range."""
    base = _randn(60, 90, seed=3)
    g = torch.stack([base * s for s in (1e30, 1e-3, 1e-30, 1.0)]).cuda()
    out = _np(_orth(g, eps=0.0))
    for i in range(4):
        assert _excess(out[i], ou.orthogonalize(_np(g[i]), eps=0.0), U) <= TOL
    # eps decides where the norm is far below it: X_0 is then nearly zero
    tiny = _np(_orth(g[2:3]))
    assert np.abs(tiny).max() <= 485 * 1e-22


def test_zero_nan_and_infinite_matrices_leave_the_others():
    g = _randn(5, 70, 130, seed=4).cuda()
    clean = _orth(g)
    g[0] = 0
    g[2, 3, 4] = float("nan")
    g[3, 69, 129] = float("inf")
    out = _orth(g)
    assert not out[0].any()
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
    assert torch.equal(out[1], clean[1]) and torch.equal(out[4], clean[4])


def test_in_place_and_views():
    """Gate columns of gate | up tensors: the up columns stay; out may be g."""
    n, rows, cols = 3, 65, 50
    for dt in (F32, BF16):
        full = _randn(n, rows, 2 * cols, seed=5).to(dt).cuda()
        ref = _orth(full[:, :, cols:].contiguous(), dt)
        work = full.clone()
        moe.moe_orthogonalize(work[:, :, cols:], work[:, :, cols:], _ws(n, rows, cols))
        torch.cuda.synchronize()
        assert torch.equal(work[:, :, cols:], ref)
        assert torch.equal(work[:, :, :cols], full[:, :, :cols])
    one = _randn(rows, cols, seed=6).cuda()  # a single matrix
    out = torch.empty_like(one)
    moe.moe_orthogonalize(one, out, _ws(1, rows, cols))
    assert _excess(_np(out), ou.orthogonalize(_np(one)), U) <= TOL
    odd = torch.full((n * rows * cols + 3,), 9.0, device="cuda")  # starts at an odd element
    v = odd[1:1 + n * rows * cols].view(n, rows, cols)
    v.copy_(full[:, :, cols:].float())
    ref = _orth(v.clone())
    moe.moe_orthogonalize(v, v, _ws(n, rows, cols))
    torch.cuda.synchronize()
    assert torch.equal(v, ref) and odd[0] == 9 and (odd[-2:] == 9).all()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("g_dtype,w_dtype", [(F32, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (2, 40, 72), (3, 130, 64), (1, 257, 100)])
def test_muon_update(n, rows, cols, g_dtype, w_dtype, nesterov):
    print(f"[muon] n={n} {rows}x{cols} {g_dtype} {w_dtype} {nesterov}", flush=True)
    g = (_randn(n, rows, cols, seed=1) * 1e-2).to(g_dtype).cuda()
    m0 = (_randn(n, rows, cols, seed=2) * 1e-2).cuda()
    w0 = (_randn(n, rows, cols, seed=3) * 0.05).to(w_dtype).cuda()
    kw = dict(lr=0.02, mu=0.9, weight_decay=0.1, scale=1.5, nesterov=nesterov)
    m, w, ws = m0.clone(), w0.clone(), _ws(n, rows, cols)
    moe.moe_muon_update(g, m, w, ws, **kw)
    torch.cuda.synchronize()
    for i in range(n):
        rm, rw = ou.muon_update(_np(g[i]), _np(m0[i]), _np(w0[i]), **kw)
        gi, mi, wi = _np(g[i]), _np(m0[i]), _np(w0[i])
        # mu is rounded to fp32 on the way, then one or two roundings
        assert np.all(np.abs(_np(m[i]) - rm) <= 3 * U * (np.abs(gi) + np.abs(mi)))
        excess = np.maximum(np.abs(_np(w[i]) - rw) - (HALF[w_dtype] + U) * np.abs(rw)
                            - 4 * U * np.abs(wi), 0.0)
        # fp32 roundings of lr, scale and decay: 4 units of the update too
        assert np.linalg.norm(excess) <= 0.02 * 1.5 * (TOL + 4 * U * np.sqrt(min(rows, cols)))


@pytest.mark.parametrize("n,rows,cols", MANY)
def test_muon_many_matrices(n, rows, cols):
    """bf16 weights: the last product's operands are rounded to fp16, an error of
    at most 2^-11 of |Q| |X| per entry: |Q|_2 <= 11.9, |X|_F <= 1.21 sqrt(m)."""
    print(f"[muon] n={n} {rows}x{cols}", flush=True)
    gen = torch.Generator("cuda").manual_seed(n)
    g, m, w = (torch.randn(n, rows, cols, device="cuda", generator=gen) * s
               for s in (1e-2, 1e-2, 0.05))
    w = w.to(BF16)
    keep = [0, n // 2, n - 1]
    old = [(_np(g[i]), _np(m[i]), _np(w[i])) for i in keep]
    kw = dict(lr=0.02, mu=0.9, weight_decay=0.1, scale=1.5)
    moe.moe_muon_update(g, m, w, _ws(n, rows, cols), **kw)
    torch.cuda.synchronize()
    tol = 0.02 * 1.5 * (TOL + 11.9 * 1.21 * np.sqrt(min(rows, cols)) * 2.0 ** -11)
    for i, (gi, mi, wi) in zip(keep, old):
        rm, rw = ou.muon_update(gi, mi, wi, **kw)
        assert np.all(np.abs(_np(m[i]) - rm) <= 3 * U * (np.abs(gi) + np.abs(mi)))
        assert _excess(_np(w[i]), rw, HALF[BF16] + U) <= tol


def test_muon_views_and_no_gradient():
    n, rows, cols = 2, 48, 80
    full = {k: _randn(n, rows, 2 * cols, seed=i).cuda() for i, k in enumerate("gmw")}
    full["g"][1] = 0
    full["m"][1] = 0
    ref = {k: full[k][:, :, :cols].contiguous() for k in "gmw"}
    old = {k: v.clone() for k, v in full.items()}
    kw = dict(lr=0.1, weight_decay=0.5, scale=0.3)
    moe.moe_muon_update(ref["g"], ref["m"], ref["w"], _ws(n, rows, cols), **kw)
    moe.moe_muon_update(*(full[k][:, :, :cols] for k in "gmw"), _ws(n, rows, cols), **kw)
    torch.cuda.synchronize()
    for k in "gmw":
        assert torch.equal(full[k][:, :, :cols], ref[k])
        assert torch.equal(full[k][:, :, cols:], old[k][:, :, cols:])
    assert torch.equal(full["g"], old["g"])
    keep = torch.tensor(1.0 - np.float32(0.1) * np.float32(0.5), dtype=F32)
    assert torch.allclose(ref["w"][1], old["w"][1, :, :cols] * keep.cuda(), rtol=2e-7, atol=0)


def test_same_bits_on_another_stream_and_in_a_graph():
    n, rows, cols = 4, 200, 333
    g = _randn(n, rows, cols, seed=8).cuda()
    m0, w0 = _randn(n, rows, cols, seed=9).cuda(), _randn(n, rows, cols, seed=10).to(BF16).cuda()
    m, w, out, ws = m0.clone(), w0.clone(), torch.empty_like(g), _ws(n, rows, cols)

    def step():
        moe.moe_orthogonalize(g, out, ws)
        moe.moe_muon_update(g, m, w, ws, lr=0.01)

    def reset():
        m.copy_(m0)
        w.copy_(w0)
        out.zero_()

    step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (out, m, w)]
    reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, (out, m, w)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        reset()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, (out, m, w)))
        moe.moe_orthogonalize(m0, out, ws)  # eager work between replays, the same workspace
        torch.cuda.synchronize()
    # a workspace larger than needed and dirty gives the same bits
    big = torch.full((ws.numel() + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    out2 = torch.empty_like(out)
    moe.moe_orthogonalize(g, out2, big)
    assert torch.equal(out2, ref[0])


@pytest.mark.parametrize("n,rows,cols", [(5, 120, 300), (300, 64, 40)])
def test_short_sides_in_a_graph_and_two_at_once(n, rows, cols):
    print(f"[orth] graph n={n} {rows}x{cols}", flush=True)
    g, g2 = _randn(n, rows, cols, seed=21).cuda(), _randn(n, rows, cols, seed=22).cuda()
    m0, w0 = _randn(n, rows, cols, seed=23).cuda(), _randn(n, rows, cols, seed=24).cuda()
    m, w, ws, ws2 = m0.clone(), w0.clone(), _ws(n, rows, cols), _ws(n, rows, cols)
    moe.moe_muon_update(g, m, w, ws, lr=0.02)
    ref, ref2 = [m.clone(), w.clone()], _orth(g2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_muon_update(g, m, w, ws, lr=0.02)
    side, out2 = torch.cuda.Stream(), torch.empty_like(g2)
    for _ in range(3):
        m.copy_(m0)
        w.copy_(w0)
        out2.zero_()
        torch.cuda.synchronize()
        graph.replay()
        moe.moe_orthogonalize(g2, out2, ws2, stream=side.cuda_stream)  # beside it
        torch.cuda.synchronize()
        assert torch.equal(m, ref[0]) and torch.equal(w, ref[1]) and torch.equal(out2, ref2)
