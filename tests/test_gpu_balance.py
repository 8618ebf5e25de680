"""Balance loss, its gradient and the dense router backward
(include/moe_balance.h) on the GPU against the numpy oracle in 64 bits.

Bounds: a softmax in fp32 (exp of a difference, itself rounded: |z - max| 2^-24
+ a few units; E additions; one division) is within (E + 64) 2^-24 of each p
for logits within 30 of each other; sums over tokens add one rounding each."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from oracle import fp8_ckpt_balance_oracle as fo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


def run_loss(z, topk, coef, mask=None):
    T, E = z.shape
    counts = torch.full((E,), -5, dtype=torch.int32, device="cuda")
    tokens = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    prob, loss = torch.full((E,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda")
    ws = torch.full((max(256, moe.moe_balance_loss_workspace_size(T, E)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss(z, topk, coef, counts, tokens, prob, loss, ws, mask=mask)
    return counts, tokens, prob, loss


def case(T, E, k, dtype=torch.float32, padded=0.3, seed=0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)).to(dtype)
    topk = torch.topk(z.float(), k, 1).indices.int()
    mask = (torch.rand(T, generator=g) >= padded).to(torch.uint8)
    return z, topk, mask, torch.randn(T, k, generator=g)


SIZES = [(1, 1, 1), (1, 8, 2), (7, 5, 3), (256, 8, 2), (300, 16, 4), (1000, 17, 2), (33, 64, 6),
         (2050, 100, 8), (700, 128, 8), (513, 256, 8), (40, 500, 16), (65, 1000, 3), (9, 1024, 16)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_loss_and_gradient(T, E, k, dtype):
    z, topk, mask, dlogit = case(T, E, k, dtype, seed=T + E)
    coef = 0.03
    for m in (None, mask):
        mg = None if m is None else m.cuda()
        mn = None if m is None else m.numpy()
        counts, tokens, prob, loss = run_loss(z.cuda(), topk.cuda(), coef, mg)
        rc, rn, rp, rl = fo.balance_loss(z.double().numpy(), topk.numpy(), coef, mn)
        assert np.array_equal(counts.cpu().numpy(), rc) and int(tokens) == rn
        tol = (E + 64 + T) * U
        assert (np.abs(prob.cpu().double().numpy() - rp) <= tol * rp).all()
        assert abs(float(loss) - rl) <= (tol + U) * rl
        dlogits = torch.full((T, E), 9.0, device="cuda")
        dloss = torch.tensor([1.5], device="cuda")
        moe.moe_balance_loss_backward(z.cuda(), topk.cuda(), coef, counts, tokens, dloss, dlogits,
                                      mask=mg, dlogit=dlogit.cuda())
        ref = fo.balance_backward(z.double().numpy(), coef, k, rc, rn, 1.5, mn, topk.numpy(),
                                  dlogit.double().numpy())
        top = 1.5 * coef * E / (k * max(rn, 1) ** 2) * rc.max()  # |f| and |sum p f| at most
        bound = 2 * top * (2 * E + 128) * U + np.abs(ref) * 2 * U + 1e-30
        assert (np.abs(dlogits.cpu().double().numpy() - ref) <= bound).all()


def test_plain_gradient_without_topk_part_and_dloss():
    z, topk, _, _ = case(50, 12, 2, seed=3)
    counts, tokens, _, _ = run_loss(z.cuda(), topk.cuda(), 0.5)
    d = torch.empty(50, 12, device="cuda")
    moe.moe_balance_loss_backward(z.cuda(), topk.cuda(), 0.5, counts, tokens, None, d)
    ref = fo.balance_backward(z.double().numpy(), 0.5, 2, counts.cpu().numpy(), 50)
    assert np.abs(d.cpu().double().numpy() - ref).max() <= 1e-6 * np.abs(ref).max()


def test_counts_of_a_whole_batch_from_two_ranks():
    """Added counts, tokens and sums give the gradient of the joint loss."""
    z, topk, mask, _ = case(200, 24, 3, seed=5)
    coef = 0.1
    half = [(z[s].contiguous().cuda(), topk[s].contiguous().cuda(), mask[s].contiguous().cuda())
            for s in (slice(0, 90), slice(90, 200))]
    parts = [run_loss(a, b, coef, m) for a, b, m in half]
    counts, tokens, prob = (parts[0][i] + parts[1][i] for i in range(3))
    rc, rn, rp, rl = fo.balance_loss(z.double().numpy(), topk.numpy(), coef, mask.numpy())
    assert np.array_equal(counts.cpu().numpy(), rc) and int(tokens) == rn
    joint = coef * 24 / (3 * rn ** 2) * float((counts.double() * prob.double()).sum())
    assert abs(joint - rl) <= 1e-5 * rl
    ref = fo.balance_backward(z.double().numpy(), coef, 3, rc, rn, 1.0, mask.numpy())
    got = []
    for a, b, m in half:
        d = torch.empty(a.shape, device="cuda")
        moe.moe_balance_loss_backward(a, b, coef, counts, tokens, None, d, mask=m)
        got.append(d.cpu().double().numpy())
    assert np.abs(np.concatenate(got) - ref).max() <= 1e-5 * np.abs(ref).max()


def test_dropped_slots_double_choices_and_no_tokens():
    z, topk, _, dlogit = case(30, 8, 3, seed=6)
    topk[0] = torch.tensor([-1, 8, 2 ** 31 - 1])
    topk[1] = torch.tensor([4, 4, 4])
    counts, tokens, prob, loss = run_loss(z.cuda(), topk.cuda(), 0.2)
    rc, rn, rp, rl = fo.balance_loss(z.double().numpy(), topk.numpy(), 0.2)
    assert np.array_equal(counts.cpu().numpy(), rc) and int(tokens) == rn == 30
    assert abs(float(loss) - rl) <= 1e-5 * rl
    d = torch.empty(30, 8, device="cuda")
    moe.moe_balance_loss_backward(z.cuda(), topk.cuda(), 0.2, counts, tokens, None, d,
                                  dlogit=dlogit.cuda())
    ref = fo.balance_backward(z.double().numpy(), 0.2, 3, rc, rn, 1.0, None, topk.numpy(),
                              dlogit.double().numpy())
    assert np.abs(d.cpu().double().numpy() - ref).max() <= 1e-5
    none = torch.zeros(30, dtype=torch.bool, device="cuda")
    counts, tokens, prob, loss = run_loss(z.cuda(), topk.cuda(), 0.2, none)
    assert int(counts.abs().sum()) == 0 and int(tokens) == 0
    assert float(prob.abs().sum()) == 0 and float(loss) == 0
    moe.moe_balance_loss_backward(z.cuda(), topk.cuda(), 0.2, counts, tokens, None, d, mask=none)
    assert (d == 0).all()
    empty = torch.empty(0, 8, device="cuda")
    counts, tokens, prob, loss = run_loss(empty, torch.empty(0, 3, dtype=torch.int32,
                                                             device="cuda"), 0.2)
    assert int(counts.abs().sum()) == 0 and int(tokens) == 0 and float(loss) == 0
    assert float(prob.abs().sum()) == 0


def test_masked_rows_and_infinite_logits():
    """NaN in rows that do not count is not looked at; -inf is an expert that
    is not offered, and a row of -inf alone adds nothing."""
    z, topk, _, _ = case(40, 20, 2, seed=7)
    mask = torch.ones(40, dtype=torch.uint8)
    mask[[3, 39]] = 0
    z[3], z[39] = float("nan"), float("inf")
    z[5, :15] = float("-inf")
    topk[5] = torch.tensor([16, 17])
    z[6] = float("-inf")
    z[7] = torch.finfo(torch.float32).min
    counts, tokens, prob, loss = run_loss(z.cuda(), topk.cuda(), 0.2, mask.cuda())
    rc, rn, rp, rl = fo.balance_loss(z.double().numpy(), topk.numpy(), 0.2, mask.numpy())
    assert np.array_equal(counts.cpu().numpy(), rc) and int(tokens) == rn == 38
    assert (np.abs(prob.cpu().double().numpy() - rp) <= 1e-5 * rp).all()
    assert abs(float(loss) - rl) <= 1e-5 * rl
    d = torch.empty(40, 20, device="cuda")
    moe.moe_balance_loss_backward(z.cuda(), topk.cuda(), 0.2, counts, tokens, None, d,
                                  mask=mask.cuda())
    d = d.cpu().numpy()
    assert np.isfinite(d).all()
    assert (d[[3, 39, 6]] == 0).all() and (d[5, :15] == 0).all()


def test_same_bits_every_call_and_graph_replays():
    z, topk, mask, dlogit = (t.cuda() for t in case(5000, 128, 8, seed=8))
    E, T = 128, 5000
    counts, tokens = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(
        1, dtype=torch.int32, device="cuda")
    prob, loss = torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
    x = torch.randn(T, 192, device="cuda").bfloat16()
    w = torch.randn(E, 192, device="cuda")
    d, dx, dw = torch.empty(T, E, device="cuda"), torch.empty(T, 192, device="cuda"), torch.empty(
        E, 192, device="cuda")
    ws = moe.workspace(max(moe.moe_balance_loss_workspace_size(T, E),
                           moe.moe_router_backward_dense_workspace_size(T, E, 192)))

    def step():
        moe.moe_balance_loss(z, topk, 0.01, counts, tokens, prob, loss, ws, mask=mask)
        moe.moe_balance_loss_backward(z, topk, 0.01, counts, tokens, None, d, mask=mask,
                                      dlogit=dlogit)
        moe.moe_router_backward_dense(d, x, w, dx, dw, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        z.copy_(torch.randn(T, E, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (counts, tokens, prob, loss, d, dx, dw)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (counts, tokens, prob, loss, d, dx, dw)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,D", [(1, 1, 64), (3, 8, 128), (65, 5, 192), (256, 8, 128),
                                   (1000, 17, 320), (2500, 64, 256), (700, 128, 448),
                                   (300, 1000, 64), (4097, 130, 64), (130, 257, 320),
                                   (64, 600, 256), (3, 1024, 448), (8200, 300, 320)])
def test_router_dense(T, E, D, dtype):
    g = torch.Generator().manual_seed(T + E + D)
    dz = torch.randn(T, E, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
    x, w = torch.randn(T, D, generator=g).to(dtype), torch.randn(E, D, generator=g)
    base = torch.randn(T, D, generator=g)
    n = moe.moe_router_backward_dense_workspace_size(T, E, D)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    dx, dw = torch.full((T, D), 3.0, device="cuda"), torch.full((E, D), 3.0, device="cuda")
    moe.moe_router_backward_dense(dz.cuda(), x.cuda(), w.cuda(), dx, dw, ws)
    a, b, c = dz.double().numpy(), x.double().numpy(), w.double().numpy()
    rx, rw = a @ c, a.T @ b
    # products and sums in fp32 (or as exact parts of them): one rounding each
    ex = np.abs(a) @ np.abs(c) * (E + 8) * U
    ew = np.abs(a).T @ np.abs(b) * (T + 8) * U
    assert (np.abs(dx.cpu().double().numpy() - rx) <= ex).all()
    assert (np.abs(dw.cpu().double().numpy() - rw) <= ew).all()
    acc = base.cuda()
    moe.moe_router_backward_dense(dz.cuda(), x.cuda(), w.cuda(), acc, None, None, accumulate=True)
    rx = rx + base.double().numpy()
    assert (np.abs(acc.cpu().double().numpy() - rx) <= ex + np.abs(rx) * U).all()
    dw2 = torch.empty(E, D, device="cuda")
    moe.moe_router_backward_dense(dz.cuda(), x.cuda(), w.cuda(), None, dw2, ws)
    assert torch.equal(dw, dw2)


def test_router_dense_without_tokens():
    dw = torch.full((8, 64), 3.0, device="cuda")
    moe.moe_router_backward_dense(torch.empty(0, 8, device="cuda"),
                                  torch.empty(0, 64, device="cuda"),
                                  torch.ones(8, 64, device="cuda"), None, dw, None)
    assert (dw == 0).all()
