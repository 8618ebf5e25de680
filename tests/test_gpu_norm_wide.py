"""Layer norm of rows far from zero, beside the widths where the kernels change
(16384 values fill the registers of a row's threads, wider ones take a loop).

Tolerances, with u = 2^-24. The mean of a row is summed from vectors of 4 or 8
values, each vector off by at most 3 u of its sum, independent of the others,
in fp64 from there: for a constant row every vector's sum is exact (but the
last, shorter one's: 3 u / D of the mean), so the mean is the constant and y is
beta, bit for bit. For others the vectors' errors average to 3 u |mean| /
sqrt(3 D / 8), 6 of which are below u |mean| / 4 from D = 13824 on, and the mean
rounds once, u |mean|: at most 1.25 u |mean|.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from oracle import norm_update_oracle as ou

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
WIDTHS = [16384, 16385, 16391, 40000, 262144]


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_constant_rows(D, dtype):
    print(f"[norm] constant D={D} {dtype}", flush=True)
    values = torch.tensor([1000.1, 100.1, -0.3, 77777.7]).to(DT[dtype])
    x = values[:, None].expand(4, D).contiguous().cuda()
    beta = torch.randn(D, generator=torch.Generator().manual_seed(0)).cuda()
    y, (mean, rstd) = torch.full_like(x, 7.0), torch.empty(2, 4, device="cuda")
    moe.moe_layer_norm(x, None, beta, 1e-5, y, mean, rstd)
    torch.cuda.synchronize()
    assert torch.equal(mean.cpu(), values.float())
    assert torch.equal(y, beta.to(DT[dtype]).expand(4, D))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_rows_far_from_zero(D, dtype):
    print(f"[norm] far D={D} {dtype}", flush=True)
    dt = DT[dtype]
    spread = 0.1 if dtype == "f32" else 20.0  # bf16 keeps 1000 in steps of 4
    x = 1000.1 + spread * torch.randn(3, D, generator=torch.Generator().manual_seed(D))
    x = x.to(dt).cuda()
    y, (mean, rstd) = torch.full_like(x, 7.0), torch.empty(2, 3, device="cuda")
    moe.moe_layer_norm(x, None, None, 1e-5, y, mean, rstd)
    torch.cuda.synchronize()
    ry, rm, rr = ou.layer_norm(_np(x))
    em = 1.25 * U * np.abs(rm)
    assert np.all(np.abs(_np(mean) - rm) <= em)
    # Squares of the centred values, off by (x - mean) u and by em, in sums of
    # at most 300 roundings (all terms are positive); half of it for rstd.
    ev = 150 * U + 4 * U + (em * rr) ** 2
    assert np.all(np.abs(_np(rstd) - rr) <= rr * ev)
    tol = (em * rr)[:, None] + np.abs(ry) * (ev[:, None] + 3 * U) + HALF[dt] * np.abs(ry)
    assert np.all(np.abs(_np(y) - ry) <= tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [8, 300, 1031, 2048, 9001, 16391])
def test_sums_past_the_range(D, dtype):
    """Values whose mean is in fp32's range and whose sums are not."""
    print(f"[norm] large D={D} {dtype}", flush=True)
    values = torch.tensor([2.0 ** 122, -2.0 ** 125]).to(DT[dtype])
    x = values[:, None].expand(2, D).contiguous().cuda()
    y, (mean, rstd) = torch.full_like(x, 7.0), torch.empty(2, 2, device="cuda")
    moe.moe_layer_norm(x, None, None, 1e-5, y, mean, rstd)
    torch.cuda.synchronize()
    assert torch.equal(mean.cpu(), values.float()) and not y.any()
    # eps rounded to fp32, a root and a division: 2 u of 1 / sqrt(eps)
    assert np.all(np.abs(_np(rstd) * np.sqrt(1e-5) - 1) <= 3 * U)


@pytest.mark.parametrize("gamma", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [63, 300, 1031, 9001, 16391, 40001])
def test_backward_of_large_constant_rows(D, dtype, gamma):
    """mean rstd leaves fp32's range, (x - mean) rstd = 0 does not: the places of
    the last vector past D add nothing, and dx = rstd (g - mean(g))."""
    print(f"[norm] backward of constant rows D={D} {dtype} {gamma}", flush=True)
    dt, gen = DT[dtype], torch.Generator().manual_seed(D)
    x = torch.tensor([2.0 ** 122, -2.0 ** 125])[:, None].expand(2, D).contiguous().to(dt).cuda()
    gm = (1 + 0.2 * torch.randn(D, generator=gen)).cuda() if gamma else None
    dy = torch.randn(2, D, generator=gen).to(dt).cuda()
    y, dx = torch.empty_like(x), torch.full_like(x, 7.0)
    mean, rstd = torch.empty(2, 2, device="cuda")
    dgamma, dbeta = torch.full((2, D), 7.0, device="cuda")
    moe.moe_layer_norm(x, gm, None, 1e-5, y, mean, rstd)
    moe.moe_layer_norm_backward(x, dy, gm, mean, rstd, None, dx, dgamma, dbeta,
                                moe.workspace(moe.moe_layer_norm_backward_workspace_size(2, D)))
    torch.cuda.synchronize()
    assert not y.any() and not dgamma.any()
    g = _np(dy) * (_np(gm) if gamma else 1.0)
    ref = _np(rstd)[:, None] * (g - g.mean(1, keepdims=True))
    # dy gamma and the difference round once each, their mean at most 300 times
    tol = _np(rstd)[:, None] * (3 * U * np.abs(g) + 300 * U * np.abs(g).mean(1, keepdims=True))
    assert np.all(np.abs(_np(dx) - ref) <= tol + (HALF[dt] + 2 * U) * np.abs(ref))
    assert np.all(np.abs(_np(dbeta) - _np(dy).sum(0)) <= 2 * U * np.abs(_np(dy)).sum(0))
