"""FP8 with block scales (include/moe_fp8.h) on the GPU against the numpy
oracle: codes and scales bit by bit, products within the instruction's bound.

The bound of a product: a block's 128 exact products are summed inside the
matrix instruction with at most 2^-10 of the sum of their magnitudes lost;
blocks are scaled and added in fp32 (one rounding of the scale's product, one
FMA a block: (K/128 + 1) 2^-24 of the magnitudes); the result is rounded once
to its type."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from oracle import fp8_ckpt_balance_oracle as fo
from oracle import moe_oracle as om

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


def mixed_rows(rows, K, seed, dtype):
    """Rows whose blocks span many magnitudes, with blocks of zeros, of equal
    magnitudes, of subnormals."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g)
    nb = -(-K // 64)
    x = x * torch.exp2(torch.randint(-40, 40, (rows, nb), generator=g).float()
                       ).repeat_interleave(64, 1)[:, :K]
    x[0, :64] = 0.0
    if rows > 4:
        x[1, :64] = torch.linspace(-1, 1, 64) * 2.0 ** 12
        x[2, :K] = 2.0 ** -130 * torch.arange(1, K + 1).float()
        x[3, :64] = -0.0
        x[4, :K] = 448.0 * torch.where(torch.rand(K, generator=g) < 0.5, 1.0, -1.0)
    return x.to(dtype)


def quantize(x):
    rows, K = x.shape
    codes = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(-(-K // 128), rows, device="cuda")
    moe.moe_fp8_quantize_rows(x.cuda(), codes, scales)
    return codes, scales


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(1, 64), (37, 128), (300, 1088), (16, 512), (17, 4096),
                                    (129, 576), (33, 7232)])
def test_quantize_rows_bit_exact(rows, K, dtype):
    x = mixed_rows(rows, K, rows + K, dtype)
    codes, scales = quantize(x)
    want_c, want_s = fo.fp8_rows(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_rows_with_nan_and_infinity(dtype):
    x = torch.randn(5, 384, generator=torch.Generator().manual_seed(0))
    x[0, 3], x[1, 130], x[2, 383], x[3, 0] = float("nan"), float("inf"), float("-inf"), 3e38
    x = x.to(dtype)
    codes, scales = quantize(x)
    y = fo.fp8_row_values(codes.cpu().numpy(), scales.cpu().numpy())
    bad = np.zeros((5, 3), bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert np.array_equal(np.isnan(y), np.repeat(bad, 128, 1))
    ref = fo.fp8_row_values(*fo.fp8_rows(x.float().numpy()))
    assert np.array_equal(y[~np.isnan(y)], ref[~np.isnan(ref)])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,K,N", [(1, 64, 64), (3, 128, 320), (2, 448, 128), (5, 192, 576)])
def test_pack_weights_bit_exact(n, K, N, dtype):
    g = torch.Generator().manual_seed(n + K + N)
    w = torch.randn(n, K, N, generator=g) * torch.exp2(
        torch.randint(-20, 20, (n, 1, N // 64), generator=g).float()).repeat_interleave(64, 2)
    w[0, :64, :64] = 0
    w = w.to(dtype)
    codes, scales = moe.pack_expert_weights_fp8(w.cuda())
    want_c, want_s = fo.fp8_weights(w.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)


class Product:
    """Operands of a product, on both sides."""

    def __init__(self, counts, K, N, cap=None, seed=0):
        n, rows = len(counts), int(sum(counts))
        self.cap = rows if cap is None else cap
        g = np.random.default_rng(seed)
        x = (g.normal(size=(self.cap, K)) * np.exp(g.normal(size=(self.cap, 1)))).astype(np.float32)
        w = (g.normal(size=(n, K, N)) * 0.05).astype(np.float32)
        self.n, self.rows = n, rows
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.xq, self.xs = fo.fp8_rows(x)
        self.wq, self.ws = fo.fp8_weights(w)
        y, mag = fo.grouped(fo.fp8_row_values(self.xq, self.xs),
                            fo.fp8_weight_values(self.wq, self.ws), self.off)
        self.y = y
        self.err = mag * (2.0 ** -10 + (K / 128 + 2) * 2.0 ** -24)
        self.gpu = [torch.from_numpy(np.ascontiguousarray(a)).cuda()
                    for a in (self.xq, self.xs, self.off, self.wq, self.ws)]


def check_down(p, K, N, half, offsets=True):
    d = moe.make_desc(T=p.cap, D=N, E=p.n, top_k=1, I=K, y_fp16=half)
    dt = torch.float16 if half else torch.float32
    out = torch.full((p.cap, N), -7.0, dtype=dt, device="cuda")
    xq, xs, off, wq, ws = p.gpu
    moe.moe_expert_down_fp8(d, p.n, K, p.cap, xq, xs, off if offsets else None, wq, ws, out)
    y = out.cpu().double().numpy()
    u = 2.0 ** -11 if half else 2.0 ** -24
    assert (np.abs(y - p.y)[:p.rows] <= (p.err + u * np.abs(p.y) + 2.0 ** -25)[:p.rows]).all()
    assert (y[p.rows:] == -7.0).all()


def check_gate_up(p, K, I):
    d = moe.make_desc(T=p.cap, D=K, E=p.n, top_k=1, I=I)
    out = torch.full((p.cap, I), -7.0, dtype=torch.bfloat16, device="cuda")
    xq, xs, off, wq, ws = p.gpu
    moe.moe_expert_gate_up_fp8(d, p.n, I, p.cap, xq, xs, off, wq, ws, out)
    h = out.cpu().double().numpy()
    g, u = p.y[:, :I], p.y[:, I:]
    eg, eu = p.err[:, :I], p.err[:, I:]
    ref = fo.silu(g) * u
    # |SiLU'| <= 1.1; SiLU itself in fp32 from exp2 and rcp (2^-20); bf16
    bound = (1.1 * eg * (np.abs(u) + eu) + np.abs(fo.silu(g)) * eu
             + (2.0 ** -8 + 2.0 ** -19) * np.abs(ref) + 1e-30)
    assert (np.abs(h - ref)[:p.rows] <= bound[:p.rows]).all()
    assert (h[p.rows:] == -7.0).all()


COUNTS = [
    ([1], None), ([5], 9), ([0, 1, 0], None), ([3, 0, 17, 1, 0], 30), ([16, 15, 33], None),
    ([64, 65, 1, 0, 127], 300), ([200, 3, 260], None), ([0, 513, 31], 600), ([255, 257], None),
]


@pytest.mark.parametrize("counts,cap", COUNTS)
@pytest.mark.parametrize("K,N", [(64, 64), (192, 320), (512, 256), (1088, 448)])
def test_down_ragged(counts, cap, K, N):
    p = Product(counts, K, N, cap, seed=len(counts) + K)
    check_down(p, K, N, half=K % 128 == 0)


@pytest.mark.parametrize("counts,cap", COUNTS)
@pytest.mark.parametrize("K,I", [(64, 64), (192, 192), (512, 256), (1088, 320)])
def test_gate_up_ragged(counts, cap, K, I):
    check_gate_up(Product(counts, K, 2 * I, cap, seed=len(counts) + I), K, I)


@pytest.mark.parametrize("half", [False, True])
def test_down_without_offsets_and_both_types(half):
    for rows in (1, 40, 300):
        p = Product([rows], 384, 576, seed=rows)
        check_down(p, 384, 576, half, offsets=False)


def test_down_many_experts_and_long_k():
    p = Product([i % 3 for i in range(130)], 128, 128, 140, seed=1)
    check_down(p, 128, 128, False)
    p = Product([7, 90], 8256, 64, seed=2)   # 65 blocks: past 64 steps
    check_down(p, 8256, 64, False)


def test_down_no_rows_anywhere():
    p = Product([0, 0, 0], 128, 64, 50, seed=1)
    check_down(p, 128, 64, False)


def test_values_of_another_expert_and_spare_rows_do_not_leak():
    """NaN codes and infinite scales next to a segment change nothing in it."""
    counts, K, N = [20, 20, 20], 192, 192
    p = Product(counts, K, N, 80, seed=4)
    xq, xs, off, wq, ws = [t.clone() for t in p.gpu]
    xq[:20], xq[40:] = 0x7F, 0x7F
    xs[:, :20], xs[:, 40:] = float("inf"), float("nan")
    wq[0], wq[2] = 0x7F, 0x7F
    d = moe.make_desc(T=80, D=N, E=3, top_k=1, I=K)
    out = torch.zeros(80, N, device="cuda")
    moe.moe_expert_down_fp8(d, 3, K, 80, xq, xs, off, wq, ws, out)
    y = out.cpu().double().numpy()[20:40]
    assert (np.abs(y - p.y[20:40]) <= p.err[20:40] + 2.0 ** -24 * np.abs(p.y[20:40])).all()
    assert np.isnan(out[:20].cpu().numpy()).all()


def test_half_outputs_saturate():
    p = Product([4], 128, 64, seed=3)
    xs = p.gpu[1] * 1e7
    d = moe.make_desc(T=4, D=64, E=1, top_k=1, I=128, y_fp16=True)
    out = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    moe.moe_expert_down_fp8(d, 1, 128, 4, p.gpu[0], xs, p.gpu[2], p.gpu[3], p.gpu[4], out)
    y = out.cpu().double().numpy()
    assert np.isfinite(y).all()
    far = np.abs(p.y) * 1e7 > 70000
    assert far.any() and (np.abs(y[far]) == 65504).all()


@pytest.mark.parametrize("counts,cap,D,I", [([3, 0, 40], 50, 192, 320), ([300, 100], None, 256, 128),
                                            ([1, 1], None, 1024, 512)])
def test_ffn_is_its_three_calls(counts, cap, D, I):
    p = Product(counts, D, 2 * I, cap, seed=9)
    g = np.random.default_rng(10)
    wd = torch.from_numpy(g.normal(size=(p.n, I, D)).astype(np.float32) * 0.05).cuda()
    dq, ds = moe.pack_expert_weights_fp8(wd)
    xq, xs, off, wq, ws = p.gpu
    for half in (False, True):
        d = moe.make_desc(T=p.cap, D=D, E=p.n, top_k=1, I=I, y_fp16=half)
        dt = torch.float16 if half else torch.float32
        y = torch.full((p.cap, D), 5.0, dtype=dt, device="cuda")
        work = torch.full((moe.moe_ffn_fp8_workspace_size(d, I, p.cap),), 0xFF, dtype=torch.uint8,
                          device="cuda")
        moe.moe_expert_ffn_fp8(d, p.n, I, p.cap, xq, xs, off, wq, ws, dq, ds, y, work)
        h = torch.zeros(p.cap, I, dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_gate_up_fp8(d, p.n, I, p.cap, xq, xs, off, wq, ws, h)
        hq, hs = quantize(h)
        y2 = torch.full((p.cap, D), 5.0, dtype=dt, device="cuda")
        moe.moe_expert_down_fp8(d, p.n, I, p.cap, hq, hs, off, dq, ds, y2)
        assert torch.equal(y, y2)


def test_graph_replays_and_another_stream():
    p = Product([30, 0, 5], 256, 256, 40, seed=5)
    d = moe.make_desc(T=40, D=256, E=3, top_k=1, I=256)
    x = torch.randn(40, 256, device="cuda").bfloat16()
    xq, xs = torch.empty_like(p.gpu[0]), torch.empty_like(p.gpu[1])
    out = torch.zeros(40, 256, device="cuda")

    def step(stream=None):
        moe.moe_fp8_quantize_rows(x, xq, xs, stream)
        moe.moe_expert_down_fp8(d, 3, 256, 40, xq, xs, p.gpu[2], p.gpu[3], p.gpu[4], out, stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn(40, 256, device="cuda").bfloat16())
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and got[:35].abs().max() > 0 and (got[35:] == 0).all()


def test_rows_past_two_to_the_31_codes():
    """600 000 rows of 4096: the last expert's segment lies 2.4e9 bytes in."""
    rows, K, N = 600_000, 4096, 64
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(300, K, device="cuda").bfloat16()
    x[-300:] = tail
    codes, scales = torch.empty(rows, K, dtype=torch.uint8, device="cuda"), None
    scales = torch.empty(K // 128, rows, device="cuda")
    moe.moe_fp8_quantize_rows(x, codes, scales)
    del x
    tq, ts = fo.fp8_rows(tail.float().cpu().numpy())
    assert np.array_equal(codes[-300:].cpu().numpy(), tq)
    assert np.array_equal(scales[:, -300:].cpu().numpy(), ts)
    w = torch.randn(2, K, N, device="cuda") * 0.02
    wq, ws = moe.pack_expert_weights_fp8(w)
    off = torch.tensor([0, rows - 300, rows], dtype=torch.int32, device="cuda")
    d = moe.make_desc(T=rows, D=N, E=2, top_k=1, I=K)
    out = torch.empty(rows, N, device="cuda")
    moe.moe_expert_down_fp8(d, 2, K, rows, codes, scales, off, wq, ws, out)
    xv = fo.fp8_row_values(tq, ts)
    wv = fo.fp8_weight_values(wq[1:].cpu().numpy(), ws[1:].cpu().numpy())[0]
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    got = out[-300:].cpu().double().numpy()
    assert (np.abs(got - ref) <= mag * (2.0 ** -10 + 40 * 2.0 ** -24)).all()
    assert (out[:-300] == 0).all()


# ---- large tiles: buffers of many rows beyond the segments choose them ----
def widened(p, cap=9000):
    """p in a buffer of cap rows, those past the segments NaN."""
    xq, xs, off, wq, ws = p.gpu
    big_q = torch.full((cap, xq.shape[1]), 0x7F, dtype=torch.uint8, device="cuda")
    big_q[:p.rows] = xq[:p.rows]
    big_s = torch.full((xs.shape[0], cap), float("nan"), device="cuda")
    big_s[:, :p.rows] = xs[:, :p.rows]
    p.cap, p.gpu = cap, [big_q, big_s, off, wq, ws]
    p.y, p.err = (np.pad(a[:p.rows], ((0, cap - p.rows), (0, 0))) for a in (p.y, p.err))
    return p


@pytest.mark.parametrize("counts,cap", COUNTS)
@pytest.mark.parametrize("K,N", [(64, 64), (192, 320), (512, 256), (1088, 448)])
def test_down_ragged_large_tiles(counts, cap, K, N):
    p = widened(Product(counts, K, N, None, seed=len(counts) + K))
    check_down(p, K, N, half=K % 128 == 0)


@pytest.mark.parametrize("counts,cap", COUNTS)
@pytest.mark.parametrize("K,I", [(64, 64), (192, 192), (512, 256), (1088, 320)])
def test_gate_up_ragged_large_tiles(counts, cap, K, I):
    check_gate_up(widened(Product(counts, K, 2 * I, None, seed=len(counts) + I)), K, I)


def test_large_tiles_many_experts_long_k_and_no_rows():
    check_down(widened(Product([i % 3 for i in range(130)], 128, 128, seed=1)), 128, 128, False)
    check_down(widened(Product([7, 90], 8256, 64, seed=2)), 8256, 64, False)
    check_down(widened(Product([0, 0, 0], 128, 64, 1, seed=1)), 128, 64, True)


def test_large_tiles_values_of_another_expert_do_not_leak():
    counts, K, N = [20, 20, 20], 192, 192
    p = widened(Product(counts, K, N, seed=4))
    xq, xs, off, wq, ws = [t.clone() for t in p.gpu]
    xq[:20], xq[40:] = 0x7F, 0x7F
    xs[:, :20], xs[:, 40:] = float("inf"), float("nan")
    wq[0], wq[2] = 0x7F, 0x7F
    d = moe.make_desc(T=p.cap, D=N, E=3, top_k=1, I=K)
    out = torch.zeros(p.cap, N, device="cuda")
    moe.moe_expert_down_fp8(d, 3, K, p.cap, xq, xs, off, wq, ws, out)
    y = out.cpu().double().numpy()[20:40]
    assert (np.abs(y - p.y[20:40]) <= p.err[20:40] + 2.0 ** -24 * np.abs(p.y[20:40])).all()
    assert np.isnan(out[:20].cpu().numpy()).all() and (out[60:] == 0).all()


def test_small_and_large_tiles_one_tile_a_cu_apart():
    """The same rows in buffers whose small tiles number one a CU, and more."""
    p = Product([100, 28], 320, 1024, seed=7)
    got = []
    for cap in (1024, 1025, 4000):   # 8 column tiles: 256 small tiles, 272, ...
        q = widened(Product([100, 28], 320, 1024, seed=7), cap)
        d = moe.make_desc(T=cap, D=1024, E=2, top_k=1, I=320)
        out = torch.zeros(cap, 1024, device="cuda")
        moe.moe_expert_down_fp8(d, 2, 320, cap, *q.gpu, out)
        got.append(out[:128].cpu().double().numpy())
        assert (out[128:] == 0).all()
    for y in got:
        assert y.shape == p.y.shape
        assert (np.abs(y - p.y) <= p.err + 2.0 ** -24 * np.abs(p.y)).all()


def test_binding_refuses_wrong_shapes():
    p = Product([4, 4], 128, 64, seed=6)
    xq, xs, off, wq, ws = p.gpu
    d = moe.make_desc(T=8, D=64, E=2, top_k=1, I=128)
    out = torch.empty(8, 64, device="cuda")
    with pytest.raises(ValueError, match="scales"):
        moe.moe_expert_down_fp8(d, 2, 128, 8, xq, xs.t().contiguous(), off, wq, ws, out)
    with pytest.raises(ValueError, match="codes"):
        moe.moe_expert_down_fp8(d, 2, 128, 9, xq, torch.empty(1, 9, device="cuda"), off, wq, ws,
                                out)
    with pytest.raises(ValueError, match="weight codes"):
        moe.moe_expert_down_fp8(d, 2, 128, 8, xq, xs, off, wq[:1], ws, out)
    with pytest.raises(ValueError, match="y_perm"):
        moe.moe_expert_down_fp8(d, 2, 128, 8, xq, xs, off, wq, ws, out.half())
    with pytest.raises(moe.MoeError, match="invalid"):
        moe.moe_fp8_quantize_rows(torch.zeros(2, 96, device="cuda"),
                                  torch.empty(2, 96, dtype=torch.uint8, device="cuda"),
                                  torch.empty(1, 2, device="cuda"))
