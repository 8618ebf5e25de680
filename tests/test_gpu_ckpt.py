"""Activation checkpoints in 8 bits (include/moe_ckpt.h) on the GPU: row codes
bit by bit against the numpy oracle; the training forward's codes against the
fp32 pre-activations that the plain training forward keeps; the backward
against the formulas in 64 bits on the kept values.

Bounds, with u = 2^-8 (bf16's rounding is at most u of the value): dgu and h
come from fp32 arithmetic on exact kept values and one rounding; dH is a bf16
product summed in fp32, (D + 2) 2^-24 of its magnitudes off."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from oracle import fp8_ckpt_balance_oracle as fo

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


def rows_of(rows, D, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, D, generator=g) * torch.exp2(
        torch.randint(-60, 60, (rows, D // 32), generator=g).float()).repeat_interleave(32, 1)
    x[0, :32] = 0
    if rows > 3:
        x[1, :32] = -0.0
        x[2, :32] = 2.0 ** -131 * torch.arange(32)
        x[3, :32] = torch.arange(32) - 15.5   # ties
    return x.to(dtype)


def save(x):
    codes = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    scales = torch.empty(x.shape[0], x.shape[1] // 32, dtype=BF, device="cuda")
    moe.moe_ckpt_save_rows(x.cuda(), codes, scales)
    return codes, scales


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("rows,D", [(1, 32), (7, 96), (300, 320), (4097, 64), (5, 7168)])
def test_save_and_restore_bit_exact(rows, D, dtype):
    x = rows_of(rows, D, rows + D, dtype)
    codes, scales = save(x)
    want_c, want_s = fo.ckpt_rows(x.float().numpy())
    assert np.array_equal(bits(scales), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    back = torch.from_numpy(fo.ckpt_values(want_c, want_s))
    for dt in (torch.float32, BF):
        out = torch.empty(rows, D, dtype=dt, device="cuda")
        moe.moe_ckpt_restore_rows(codes, scales, out)
        assert torch.equal(out.cpu(), back.to(dt))


def test_many_normal_rows_bit_exact():
    x = torch.randn(3000, 2048, generator=torch.Generator().manual_seed(1))
    for dt in (torch.float32, BF):
        codes, scales = save(x.to(dt))
        want_c, want_s = fo.ckpt_rows(x.to(dt).float().numpy())
        assert np.array_equal(bits(scales), want_s)
        assert np.array_equal(codes.cpu().numpy(), want_c)


def test_nan_and_infinity_stay_in_their_block():
    x = torch.randn(4, 96, generator=torch.Generator().manual_seed(2))
    x[0, 5], x[1, 40], x[2, 95], x[3, 0] = float("nan"), float("inf"), float("-inf"), 3e38
    for dt in (torch.float32, BF):
        codes, scales = save(x.to(dt))
        out = torch.empty(4, 96, device="cuda")
        moe.moe_ckpt_restore_rows(codes, scales, out)
        bad = np.zeros((4, 3), bool)
        bad[0, 0] = bad[1, 1] = bad[2, 2] = True
        assert np.array_equal(np.isnan(out.cpu().numpy()), np.repeat(bad, 32, 1))


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_largest_values_stay_finite(dtype):
    """A type's largest value comes back finite, in bf16 too."""
    top = torch.finfo(dtype).max
    x = torch.randn(6, 96, generator=torch.Generator().manual_seed(8)).to(dtype)
    x[0, 3], x[1, 40], x[2, 64] = top, -top, 255 * 2.0 ** 120
    x[3, :32] = torch.linspace(-1, 1, 32).double().mul(top).to(dtype)
    x[4, 0], x[5, 95] = 126.4 * 2.0 ** 121, 2.0 ** 127
    codes, scales = save(x)
    want_c, want_s = fo.ckpt_rows(x.float().numpy())
    assert np.array_equal(bits(scales), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    for dt in (torch.float32, BF):
        out = torch.empty(6, 96, dtype=dt, device="cuda")
        moe.moe_ckpt_restore_rows(codes, scales, out)
        assert torch.isfinite(out).all()
        assert torch.equal(out.cpu(), torch.from_numpy(fo.ckpt_values(want_c, want_s)).to(dt))


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_restore_through_an_index(dtype):
    rows, D, n = 50, 160, 333
    x = rows_of(rows, D, 3, dtype)
    codes, scales = save(x)
    g = torch.Generator().manual_seed(4)
    index = torch.randint(0, rows, (n,), generator=g, dtype=torch.int32)
    index[[0, 7, 332]] = torch.tensor([-1, rows, 2 ** 31 - 1], dtype=torch.int32)
    out = torch.full((n, D), -7.0, dtype=dtype, device="cuda")
    moe.moe_ckpt_restore_rows(codes, scales, out, index.cuda())
    back = torch.from_numpy(fo.ckpt_values(codes.cpu().numpy(), bits(scales))).to(dtype)
    ok = (index >= 0) & (index < rows)
    want = torch.full((n, D), -7.0, dtype=dtype)
    want[ok] = back[index[ok].long()]
    assert torch.equal(out.cpu(), want)


def test_rows_past_two_to_the_31_values():
    rows, D = 1_100_000, 2048
    x = torch.zeros(rows, D, dtype=BF, device="cuda")
    tail = rows_of(5, D, 5, BF)
    x[-5:] = tail.cuda()
    codes, scales = torch.empty(rows, D, dtype=torch.int8, device="cuda"), None
    scales = torch.empty(rows, D // 32, dtype=BF, device="cuda")
    moe.moe_ckpt_save_rows(x, codes, scales)
    want_c, want_s = fo.ckpt_rows(tail.float().numpy())
    assert np.array_equal(codes[-5:].cpu().numpy(), want_c)
    assert np.array_equal(bits(scales[-5:]), want_s)
    out = torch.ones(rows, D, dtype=BF, device="cuda")
    index = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    moe.moe_ckpt_restore_rows(codes, scales, out, index)
    back = torch.from_numpy(fo.ckpt_values(want_c, want_s)).to(BF)
    assert torch.equal(out[:5].cpu(), back.flip(0))
    assert (out[5:] == 0).all()


class Layer:
    def __init__(self, counts, D, I, cap=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.rows, self.D, self.I = len(counts), sum(counts), D, I
        self.cap = self.rows if cap is None else cap
        self.x = torch.randn(self.cap, D, generator=g).to(BF).cuda()
        self.wgu = (torch.randn(self.n, D, 2 * I, generator=g) * D ** -0.5 * 1.5).to(BF).cuda()
        self.wd = (torch.randn(self.n, I, D, generator=g) * I ** -0.5).to(BF).cuda()
        self.dy = torch.randn(self.cap, D, generator=g).to(BF).cuda()
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
        self.d = moe.make_desc(T=self.cap, D=D, E=self.n, top_k=1, I=I)

    def kept(self, fill=3):
        codes = torch.full((self.cap, 2 * self.I), fill, dtype=torch.int8, device="cuda")
        scales = torch.full((self.cap, 2 * self.I // 32), 2.0, dtype=BF, device="cuda")
        return codes, scales


CASES = [([5], 128, 64, None), ([0, 3, 0, 40, 1], 320, 192, 50), ([300, 20, 0, 90], 192, 320, None),
         ([700, 2], 256, 128, 800), ([1], 64, 64, 1)]


# Buffers of many rows choose longer row blocks (up to 320).
WIDE = [([300, 20, 0, 90], 192, 128, 30000), ([700, 2], 128, 128, 45000),
        ([1, 650, 33], 64, 192, 70000), ([0, 319, 321, 640], 64, 64, 90000)]


@pytest.mark.parametrize("counts,D,I,cap", CASES + WIDE)
def test_training_forward_codes(counts, D, I, cap):
    """y_perm is the plain training forward's bit for bit, and the codes are
    those of the fp32 G | U that it keeps."""
    L = Layer(counts, D, I, cap)
    ws = moe.workspace(moe.moe_ffn_workspace_size(L.d, I, L.cap))
    y, y8 = (torch.full((L.cap, D), 9.0, device="cuda") for _ in range(2))
    gu = torch.empty(L.cap, 2 * I, device="cuda")
    moe.moe_expert_ffn_train(L.d, L.n, I, L.cap, L.x, L.off, L.wgu, L.wd, y, gu, ws)
    codes, scales = L.kept()
    moe.moe_expert_ffn_train_ckpt(L.d, L.n, I, L.cap, L.x, L.off, L.wgu, L.wd, y8, codes, scales,
                                  ws)
    assert torch.equal(y, y8)
    want_c, want_s = fo.ckpt_rows(gu[:L.rows].cpu().numpy())
    assert np.array_equal(codes[:L.rows].cpu().numpy(), want_c)
    assert np.array_equal(bits(scales[:L.rows]), want_s)
    assert (codes[L.rows:] == 3).all() and (scales[L.rows:] == 2).all()
    h, h0 = (torch.full((L.cap, I), 5.0, dtype=torch.float16, device="cuda") for _ in range(2))
    c2, s2 = L.kept()
    moe.moe_expert_gate_up_train_ckpt(L.d, L.n, I, L.cap, L.x, L.off, L.wgu, h, c2, s2)
    moe.moe_expert_gate_up(L.d, L.n, I, L.cap, L.x, L.off, L.wgu, h0)
    assert torch.equal(h, h0) and torch.equal(c2, codes) and torch.equal(s2, scales)


def reference_backward(L, codes, scales):
    """dgu, h in float64 and dH's error, from the kept values."""
    gu = fo.ckpt_values(codes.cpu().numpy(), bits(scales)).astype(np.float64)[:L.rows]
    dy, wd = L.dy[:L.rows].double().cpu().numpy(), L.wd.double().cpu().numpy()
    off = L.off.cpu().numpy()
    dh, mag = fo.grouped(dy, wd, off)
    dg, du, h = fo.swiglu_backward(gu[:, :L.I], gu[:, L.I:], dh)
    edh = mag * (L.D + 2) * 2.0 ** -24
    eg, eu, _ = fo.swiglu_backward(gu[:, :L.I], gu[:, L.I:], edh)
    ref = np.concatenate([dg, du], 1)
    err = np.abs(np.concatenate([eg, eu], 1))
    return ref, err, h


@pytest.mark.parametrize("counts,D,I,cap", CASES + WIDE)
def test_backward_from_codes(counts, D, I, cap):
    L = Layer(counts, D, I, cap, seed=1)
    codes, scales = L.kept()
    h = torch.empty(L.cap, I, dtype=torch.float16, device="cuda")
    moe.moe_expert_gate_up_train_ckpt(L.d, L.n, I, L.cap, L.x, L.off, L.wgu, h, codes, scales)
    dgu = torch.full((L.cap, 2 * I), 6.0, dtype=BF, device="cuda")
    hb = torch.full((L.cap, I), 6.0, dtype=BF, device="cuda")
    moe.moe_expert_gate_up_backward_ckpt(L.d, L.n, I, L.cap, L.dy, L.off, L.wd, codes, scales, dgu,
                                         hb)
    ref, err, href = reference_backward(L, codes, scales)
    got, hgot = dgu.double().cpu().numpy(), hb.double().cpu().numpy()
    # one bf16 rounding, the sigmoid from exp2 and rcp (2^-20 of each term; the
    # derivative's terms s and G s (1 - s) are together at most 1.1 + |G s|)
    assert (np.abs(got[:L.rows] - ref) <= 2.0 ** -8 * np.abs(ref) + err * 1.01
            + 2.0 ** -17 * np.abs(ref).max(1, keepdims=True)).all()
    assert (np.abs(hgot[:L.rows] - href) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(href) + 1e-30).all()
    assert (got[L.rows:] == 6).all() and (hgot[L.rows:] == 6).all()


@pytest.mark.parametrize("counts,D,I,cap", CASES[1:4])
def test_ffn_backward_is_its_pieces(counts, D, I, cap):
    """dx_perm and the weight gradients are those of the plain pieces on the
    dgu and h of the checkpoint's backward, bit for bit."""
    L = Layer(counts, D, I, cap, seed=2)
    codes, scales = L.kept()
    y = torch.empty(L.cap, D, device="cuda")
    ws = moe.workspace(max(moe.moe_ffn_workspace_size(L.d, I, L.cap),
                           moe.moe_ffn_backward_workspace_size(L.d, I, L.cap)))
    moe.moe_expert_ffn_train_ckpt(L.d, L.n, I, L.cap, L.x, L.off, L.wgu, L.wd, y, codes, scales, ws)
    dx = torch.full((L.cap, D), 4.0, device="cuda")
    dwgu, dwd = torch.empty(L.n, D, 2 * I, device="cuda"), torch.empty(L.n, I, D, device="cuda")
    moe.moe_expert_ffn_backward_ckpt(L.d, L.n, I, L.cap, L.x, L.off, L.wgu, L.wd, L.dy, codes,
                                     scales, dx, dwgu, dwd, ws)
    dgu = torch.zeros(L.cap, 2 * I, dtype=BF, device="cuda")
    hb = torch.zeros(L.cap, I, dtype=BF, device="cuda")
    moe.moe_expert_gate_up_backward_ckpt(L.d, L.n, I, L.cap, L.dy, L.off, L.wd, codes, scales, dgu,
                                         hb)
    wgu2, wd2 = torch.empty_like(dwgu), torch.empty_like(dwd)
    moe.moe_expert_weight_grad(L.d, L.n, L.cap, hb, I, L.dy, D, L.off, wd2)
    moe.moe_expert_weight_grad(L.d, L.n, L.cap, L.x, D, dgu, 2 * I, L.off, wgu2)
    assert torch.equal(dwgu, wgu2) and torch.equal(dwd, wd2)
    ref, _ = fo.grouped(dgu.double().cpu().numpy()[:L.rows], L.wgu.double().cpu().numpy(),
                        L.off.cpu().numpy())
    mag = fo.grouped(np.abs(dgu.double().cpu().numpy()[:L.rows]),
                     np.abs(L.wgu.double().cpu().numpy()), L.off.cpu().numpy())[0]
    assert (np.abs(dx.double().cpu().numpy()[:L.rows] - ref) <= mag * (2 * I + 2) * 2.0 ** -24).all()
    assert (dx[L.rows:] == 4).all()
    # without dx, and on no rows at all: the weight gradients, zero
    keep = dwgu.clone()
    moe.moe_expert_ffn_backward_ckpt(L.d, L.n, I, L.cap, L.x, L.off, L.wgu, L.wd, L.dy, codes,
                                     scales, None, dwgu, dwd, ws)
    assert torch.equal(keep, dwgu)
    none = torch.zeros(L.n + 1, dtype=torch.int32, device="cuda")
    moe.moe_expert_ffn_backward_ckpt(L.d, L.n, I, 0, L.x, none, L.wgu, L.wd, L.dy, codes, scales,
                                     None, dwgu, dwd, ws)
    assert (dwgu == 0).all() and (dwd == 0).all()


def test_gradient_of_the_checkpoint_is_near_the_exact_one():
    """Keeping G | U in 8 bits moves dgu by about the codes' own error: half a
    step is 1/254 of a block's largest value, some 0.6 % of the standard
    deviation on average; two kept factors and SiLU's slope (at most 1.1) keep
    dgu within 2 % of the fp32 checkpoint's in norm."""
    L = Layer([500, 300], 512, 256, seed=3)
    ws = moe.workspace(max(moe.moe_ffn_workspace_size(L.d, L.I, L.cap),
                           moe.moe_ffn_backward_workspace_size(L.d, L.I, L.cap)))
    y, gu = torch.empty(L.cap, L.D, device="cuda"), torch.empty(L.cap, 2 * L.I, device="cuda")
    codes, scales = L.kept()
    moe.moe_expert_ffn_train(L.d, L.n, L.I, L.cap, L.x, L.off, L.wgu, L.wd, y, gu, ws)
    moe.moe_expert_ffn_train_ckpt(L.d, L.n, L.I, L.cap, L.x, L.off, L.wgu, L.wd, y, codes, scales,
                                  ws)
    grads = []
    for kept in (False, True):
        dx = torch.empty(L.cap, L.D, device="cuda")
        dwgu = torch.empty(L.n, L.D, 2 * L.I, device="cuda")
        dwd = torch.empty(L.n, L.I, L.D, device="cuda")
        if kept:
            moe.moe_expert_ffn_backward_ckpt(L.d, L.n, L.I, L.cap, L.x, L.off, L.wgu, L.wd, L.dy,
                                             codes, scales, dx, dwgu, dwd, ws)
        else:
            moe.moe_expert_ffn_backward(L.d, L.n, L.I, L.cap, L.x, L.off, L.wgu, L.wd, L.dy, dx,
                                        dwgu, dwd, ws, gu_saved=gu)
        grads.append((dx, dwgu, dwd))
    for a, b in zip(*grads):
        assert float((a - b).norm() / a.norm()) < 0.02


def test_graph_replays():
    L = Layer([40, 0, 9], 128, 64, 60, seed=4)
    codes, scales = L.kept()
    h = torch.zeros(L.cap, L.I, dtype=torch.float16, device="cuda")
    dgu = torch.zeros(L.cap, 2 * L.I, dtype=BF, device="cuda")
    hb = torch.zeros(L.cap, L.I, dtype=BF, device="cuda")

    def step():
        moe.moe_expert_gate_up_train_ckpt(L.d, L.n, L.I, L.cap, L.x, L.off, L.wgu, h, codes, scales)
        moe.moe_expert_gate_up_backward_ckpt(L.d, L.n, L.I, L.cap, L.dy, L.off, L.wd, codes,
                                             scales, dgu, hb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        L.x.copy_(torch.randn(L.cap, L.D, device="cuda").to(BF))
        dgu.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = dgu.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, dgu) and got.abs().max() > 0
