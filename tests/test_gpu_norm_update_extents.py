"""Layer norm, orthogonalisation and Muon update at the ends of what their
headers allow: tensors past 2^31 elements, matrices far apart or interleaved, the
most matrices of a call, none. The results are those of the same rows and
matrices alone, bit for bit where the sizes that choose a kernel are the same,
else within the oracle's bounds."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from oracle import norm_update_oracle as ou

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# A Frobenius norm's share, far above the 1e-5 seen at full rank and below one
# wrong entry of the matrices here.
REL = 1e-3


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _np(t):
    return t.detach().double().cpu().numpy()


def _ws(n, rows, cols):
    return moe.workspace(moe.moe_orthogonalize_workspace_size(n, rows, cols))


@pytest.mark.parametrize("rows,D", [(270000, 8000), (9, 262143), (2100000, 1031)])
def test_norm_past_two_to_the_31(rows, D):
    print(f"[norm] rows={rows} D={D}", flush=True)
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    dy = torch.empty_like(x).normal_(generator=gen)
    y, dx = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    mean, rstd = torch.empty(2, rows, device="cuda")
    dgamma, dbeta = torch.empty(2, D, device="cuda")
    ws = moe.workspace(moe.moe_layer_norm_backward_workspace_size(rows, D))
    moe.moe_layer_norm(x, None, None, 1e-5, y, mean, rstd)
    moe.moe_layer_norm_backward(x, dy, None, mean, rstd, None, dx, dgamma, dbeta, ws)
    torch.cuda.synchronize()
    for a in (0, rows // 2, rows - 3):
        part = slice(a, a + 3)
        xs, dys = x[part].clone(), dy[part].clone()
        ys, dxs, (ms, rs) = torch.empty_like(xs), torch.empty_like(xs), torch.empty(2, 3,
                                                                                device="cuda")
        moe.moe_layer_norm(xs, None, None, 1e-5, ys, ms, rs)
        moe.moe_layer_norm_backward(xs, dys, None, ms, rs, None, dxs, None, None, None)
        torch.cuda.synchronize()
        assert torch.equal(y[part], ys) and torch.equal(dx[part], dxs)
        assert torch.equal(mean[part], ms) and torch.equal(rstd[part], rs)
    # Column sums of a few columns, every row in them: at most rows + 40 roundings.
    c = torch.tensor([0, 1, D // 2, D - 1], device="cuda")
    d = dy[:, c].double()
    h = (x[:, c].double() - mean.double()[:, None]) * rstd.double()[:, None]
    assert torch.all((dbeta[c].double() - d.sum(0)).abs() <= (rows + 40) * U * d.abs().sum(0))
    tol = (rows + 40) * U * (d * h).abs().sum(0) + 3 * U * (d.abs() * (h.abs() + 1)).sum(0)
    assert torch.all((dgamma[c].double() - (d * h).sum(0)).abs() <= tol)


def test_matrices_far_apart():
    """A stride of 2^31 elements, and rows 2^24 apart: past 32 bits in both."""
    n, rows, cols = 2, 140, 200
    flat = torch.zeros((1 << 31) * 2 + 64, device="cuda")
    gen = torch.Generator("cuda").manual_seed(2)
    vals = torch.empty(n, rows, cols, device="cuda").normal_(generator=gen)
    for strides in ((1 << 31, cols + 3, 1), (cols, 1 << 24, 1)):
        print(f"[orth] strides={strides}", flush=True)
        view = flat.as_strided((n, rows, cols), strides)
        view.copy_(vals)
        ws, out = _ws(n, rows, cols), torch.empty_like(vals)
        moe.moe_orthogonalize(vals, out, ws)
        moe.moe_orthogonalize(view, view, ws)
        torch.cuda.synchronize()
        assert torch.equal(view, out)
        m, w = torch.zeros_like(vals), torch.zeros_like(vals)
        view.zero_()
        moe.moe_muon_update(vals, m, w, ws, lr=1.0)
        moe.moe_muon_update(vals, torch.zeros_like(vals), view, ws, lr=1.0)
        torch.cuda.synchronize()
        assert torch.equal(view, w)
        view.zero_()
        assert not flat[:1 << 20].any() and not flat[-(1 << 20):].any()


@pytest.mark.parametrize("n,rows,cols", [(5, 64, 48), (4, 150, 132), (3, 33, 17)])
def test_interleaved_matrices(n, rows, cols):
    """Matrix i in columns [i cols, (i + 1) cols) of one [rows, n cols] tensor:
    a stride below a matrix's own extent."""
    print(f"[orth] interleaved n={n} {rows}x{cols}", flush=True)
    for dt in (torch.float32, torch.bfloat16):
        full = torch.randn(rows, n * cols, device="cuda",
                           generator=torch.Generator("cuda").manual_seed(n)).to(dt)
        view = full.view(rows, n, cols).transpose(0, 1)
        ref, ws = torch.empty(n, rows, cols, dtype=dt, device="cuda"), _ws(n, rows, cols)
        moe.moe_orthogonalize(view.contiguous(), ref, ws)
        moe.moe_orthogonalize(view, view, ws)
        torch.cuda.synchronize()
        assert torch.equal(view, ref)


def test_most_matrices_of_a_call():
    n, rows, cols = 65535, 3, 5
    g = torch.randn(n, rows, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    out, ws = torch.full_like(g, 7.0), _ws(n, rows, cols)
    moe.moe_orthogonalize(g, out, ws)
    torch.cuda.synchronize()
    for i in (0, 1, 32768, n - 1):
        ref = ou.orthogonalize(_np(g[i]))
        assert np.linalg.norm(_np(out[i]) - ref) <= REL * np.linalg.norm(ref), i
    assert torch.isfinite(out).all() and float(out.abs().max()) < 1.3
    with pytest.raises(moe.MoeError):
        big = torch.zeros(65536, 1, 1, device="cuda")
        moe.moe_orthogonalize(big, big, ws)


def test_no_matrices():
    g = torch.empty(0, 40, 70, device="cuda")
    assert moe.moe_orthogonalize_workspace_size(0, 40, 70) == 0
    moe.moe_orthogonalize(g, g, None)
    moe.moe_muon_update(g, g.clone(), g.clone(), None, lr=0.1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("n,rows,cols", [(1, 1, 262144), (1, 262144, 3), (1, 20000, 140)])
def test_longest_sides(n, rows, cols):
    print(f"[orth] long n={n} {rows}x{cols}", flush=True)
    g = torch.randn(n, rows, cols, device="cuda",
                    generator=torch.Generator("cuda").manual_seed(rows))
    out = torch.full_like(g, 7.0)
    moe.moe_orthogonalize(g, out, _ws(n, rows, cols))
    torch.cuda.synchronize()
    ref = ou.orthogonalize(_np(g[0]))
    assert np.linalg.norm(_np(out[0]) - ref) <= REL * np.linalg.norm(ref)
