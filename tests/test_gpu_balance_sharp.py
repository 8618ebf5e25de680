"""Balance loss, its gradient and the dense router backward: bounds for each
entry that scale with its probability, and sizes at which every loop of the
kernels runs more than once.

Bounds, U = 2^-24. A probability p: its argument z - max is rounded once (U of
up to 30 here), exp and the reciprocal cost a few units, the sum E additions:
(E + 64) U of p. The gradient p (f - sum p f): f is rounded once, the sum costs
E additions more, so that it is off by p (f + sum p f) (3 E + 256) U, f = dloss
coef E / (k N^2) c, and by one rounding where dlogit is added. prob_sum: a
thread adds at most 32 tokens here (a workgroup some 8 K logits, or a 128th of
them), a workgroup nine levels, the rest is in fp64: (E + 64 + 64) U."""
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


SIZES = [(20000, 8, 8), (16400, 13, 2), (5000, 40, 6), (3000, 128, 8), (1100, 250, 3),
         (900, 256, 16), (400, 512, 8), (9000, 1024, 4), (350, 1000, 16)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_loss_and_gradient_entry_by_entry(T, E, k, dtype):
    g = torch.Generator().manual_seed(T + E + k)
    z = (torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)).to(dtype)
    topk = torch.topk(z.float(), k, 1).indices.int()
    mask = (torch.rand(T, generator=g) >= 0.2).to(torch.uint8)
    dlogit = torch.randn(T, k, generator=g) * 1e-6
    coef, dl = 0.03, 1.5
    zg, tg, mg = z.cuda(), topk.cuda(), mask.cuda()
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    tokens = torch.empty(1, dtype=torch.int32, device="cuda")
    prob, loss = torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
    ws = moe.workspace(moe.moe_balance_loss_workspace_size(T, E))
    moe.moe_balance_loss(zg, tg, coef, counts, tokens, prob, loss, ws, mask=mg)
    zn, mn = z.double().numpy(), mask.numpy()
    rc, rn, rp, rl = fo.balance_loss(zn, topk.numpy(), coef, mn)
    assert np.array_equal(counts.cpu().numpy(), rc) and int(tokens) == rn
    tol = (E + 128) * U
    assert (np.abs(prob.cpu().double().numpy() - rp) <= tol * rp).all()
    assert abs(float(loss) - rl) <= (tol + U) * rl

    p = fo.softmax(zn) * (mn != 0)[:, None]
    f = dl * coef * E / (k * float(rn) ** 2) * rc
    bound = p * (f + (p * f).sum(1, keepdims=True)) * (3 * E + 256) * U
    ref = fo.balance_backward(zn, coef, k, rc, rn, dl, mn)
    on = mn != 0
    if k < E:  # (where every token takes every expert, the load is even, the gradient 0)
        # the bound says something about nearly every entry
        assert (np.abs(ref[on]) > 10 * bound[on]).mean() > 0.9
    d = torch.empty(T, E, device="cuda")
    dloss = torch.tensor([dl], device="cuda")
    moe.moe_balance_loss_backward(zg, tg, coef, counts, tokens, dloss, d, mask=mg)
    got = d.cpu().double().numpy()
    assert (np.abs(got - ref) <= bound + 1e-37).all()
    assert (got[~on] == 0).all()
    moe.moe_balance_loss_backward(zg, tg, coef, counts, tokens, dloss, d, mask=mg,
                                  dlogit=dlogit.cuda())
    both = ref.copy()
    np.add.at(both, (np.arange(T)[:, None], topk.numpy()), dlogit.double().numpy())
    assert (np.abs(d.cpu().double().numpy() - both) <= bound + np.abs(both) * 2 * U + 1e-37).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,D", [(16400, 8, 1088), (16400, 40, 1088), (16400, 128, 1088),
                                   (16400, 200, 640), (3000, 400, 1088)])
def test_router_dense_over_many_tiles(T, E, D, dtype):
    """Every wave takes several blocks of columns, every part of dW many steps.
    An element's products and sums are each rounded once: (E + 8) and (T + 8) U
    of the magnitudes; in the mean over a matrix, where partial sums are no
    larger than the whole, 512 U of it (some 400 instructions a chain)."""
    g = torch.Generator().manual_seed(T + E)
    dz = torch.randn(T, E, generator=g) * torch.exp(0.5 * torch.randn(T, 1, generator=g))
    x, w = torch.randn(T, D, generator=g).to(dtype), torch.randn(E, D, generator=g)
    base = torch.randn(T, D, generator=g)
    ws = moe.workspace(moe.moe_router_backward_dense_workspace_size(T, E, D))
    dx, dw = torch.full((T, D), 3.0, device="cuda"), torch.full((E, D), 3.0, device="cuda")
    moe.moe_router_backward_dense(dz.cuda(), x.cuda(), w.cuda(), dx, dw, ws)
    a, b, c = dz.double().numpy(), x.double().numpy(), w.double().numpy()
    for got, ref, mag in ((dx, a @ c, np.abs(a) @ np.abs(c) * (E + 8)),
                          (dw, a.T @ b, np.abs(a).T @ np.abs(b) * (T + 8))):
        err = got.cpu().double().numpy() - ref
        assert (np.abs(err) <= mag * U).all()
        assert np.linalg.norm(err) <= 512 * U * np.linalg.norm(ref)
    acc = base.cuda()
    moe.moe_router_backward_dense(dz.cuda(), x.cuda(), w.cuda(), acc, None, None, accumulate=True)
    # one sum, rounded once: the same as adding dx behind the call
    assert torch.equal(acc, base.cuda() + dx)
