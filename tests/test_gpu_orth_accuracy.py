"""How exact the Newton-Schulz orthogonalisation and the Muon update are, on
gradients of full rank and of the low ranks that experts with few tokens have.

Tolerance. A stored value (two fp16 parts) is off by at most 2^-22 of itself,
typically 2^-24, and fp32 sums by less; a step stores and sums about six
matrices, whose errors are independent: sqrt(6) 2^-24 = 1.5e-7 of X typically.
E = 2^-21 = 4.8e-7 is allowed. The iteration amplifies an error made at step i
by at most 3.4445^(5 - i) outside the gradient's range (inside it converges),
X before step i has a Frobenius norm of at most min(3.4445^i, 1.21 sqrt(r)) for
rank r, and O one of at least 0.68 sqrt(r):
  |error|_F / |O|_F <= E sum_{i = 0..5} 3.4445^(5 - i) min(3.4445^i, 1.21 sqrt(r)) / (0.68 sqrt(r))
which is 5.1e-4 at rank 1, 2.9e-4 at 8, 1.3e-4 at 64, 8e-5 at 256. Operands
without their low parts would cost 2.7e-4 to 4.4e-4 at full rank and 3.2e-3
below it. A bf16 result adds its own rounding R (computed): where an error of
size d turns the rounding of a value, the square of the value's error grows by
at most 4 d (step / 2) + 4 d^2 for a share 2 d / step of the values, so
  |error|^2 <= R^2 + 8 |d|^2.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from oracle import norm_update_oracle as ou

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
E = 2.0 ** -21


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


def _tol(rank, steps=5):
    a, root = 3.4445, np.sqrt(rank)
    return E * sum(a ** (steps - i) * min(a ** i, 1.21 * root)
                   for i in range(steps + 1)) / (0.68 * root)


def _gradients(n, rows, cols, rank, seed):
    """X^T dY of `rank` tokens; full rank (0): of 1.5 times the short side."""
    gen = torch.Generator("cuda").manual_seed(seed)
    tokens = rank or 3 * min(rows, cols) // 2
    x = torch.randn(n, rows, tokens, device="cuda", generator=gen)
    dy = torch.randn(n, tokens, cols, device="cuda", generator=gen)
    return torch.matmul(x, dy)


def _ws(n, rows, cols):
    return moe.workspace(moe.moe_orthogonalize_workspace_size(n, rows, cols))


def _exact(g, steps=5):
    return ou.orthogonalize(g.double().cpu().numpy(), steps)


def _check(got, ref, rank, what, steps=5):
    """got [rows, cols] (fp32 or bf16) against the float64 ref."""
    tol = _tol(min(rank or min(ref.shape), *ref.shape), steps) * np.linalg.norm(ref)
    err = np.linalg.norm(got.detach().double().cpu().numpy() - ref)
    if got.dtype == BF16:
        own = np.linalg.norm(torch.from_numpy(ref).to(BF16).double().numpy() - ref)
        assert err ** 2 <= own ** 2 + 8 * tol ** 2, (what, err, own, tol)
    else:
        assert err <= tol, (what, err, tol)


# One workgroup a matrix; several; products of 64 x 64, 128 x 128 and
# 256 x 256 tiles (wide, tall); a short side of 1024.
SHAPES = [(300, 96, 100), (8, 128, 512), (3, 1001, 333), (130, 256, 512), (40, 768, 800),
          (40, 800, 768), (2, 1024, 1280)]


@pytest.mark.parametrize("rank", [0, 64, 8, 1])
@pytest.mark.parametrize("n,rows,cols", SHAPES)
def test_muon_on_bf16_weights(n, rows, cols, rank):
    """Weights that start at zero: W is the step itself, rounded once."""
    print(f"[muon] bf16 n={n} {rows}x{cols} rank={rank}", flush=True)
    g = _gradients(n, rows, cols, rank, seed=rows + rank)
    m, w = torch.zeros_like(g), torch.zeros(n, rows, cols, dtype=BF16, device="cuda")
    moe.moe_muon_update(g, m, w, _ws(n, rows, cols), lr=1.0, nesterov=False)
    torch.cuda.synchronize()
    for i in (0, n - 1):
        _check(-w[i], _exact(g[i]), rank, i)


# The same, and short sides that take a launch of their own for the Gram product
# (many matrices, a long side).
@pytest.mark.parametrize("rank", [0, 64, 8, 1])
@pytest.mark.parametrize("n,rows,cols", SHAPES + [(60, 128, 520), (2, 4200, 30)])
def test_fp32_and_bf16_results(n, rows, cols, rank):
    """moe_orthogonalize into both types, and the Muon step on fp32 weights that
    start at zero: segments of one, two and three steps, on both sides of 128."""
    print(f"[orth] n={n} {rows}x{cols} rank={rank}", flush=True)
    g = _gradients(n, rows, cols, rank, seed=rows + rank + 1)
    f, h, ws = torch.full_like(g, 7.0), torch.full_like(g, 7.0, dtype=BF16), _ws(n, rows, cols)
    moe.moe_orthogonalize(g, f, ws)
    moe.moe_orthogonalize(g, h, ws)
    m, w = torch.zeros_like(g), torch.zeros_like(g)
    moe.moe_muon_update(g, m, w, ws, lr=1.0, nesterov=False)
    torch.cuda.synchronize()
    for i in (0, n - 1):
        ref = _exact(g[i])
        for name, got in (("fp32", f[i]), ("bf16", h[i]), ("muon", -w[i])):
            _check(got, ref, rank, (name, i))


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("rank", [0, 8, 1])
@pytest.mark.parametrize("n,rows,cols", [(3, 90, 200), (2, 256, 512)])
def test_more_steps(n, rows, cols, rank, out_dtype):
    """Eight steps within the bound for eight. Sixteen: outside a low-rank
    gradient's range rounding has become as large as the result (as the header
    says), which still has no singular value above 1.21."""
    print(f"[orth] steps n={n} {rows}x{cols} rank={rank} {out_dtype}", flush=True)
    g = _gradients(n, rows, cols, rank, seed=rows + rank + 2)
    out = torch.empty_like(g, dtype=out_dtype)
    moe.moe_orthogonalize(g, out, _ws(n, rows, cols), steps=8)
    for i in (0, n - 1):
        _check(out[i], _exact(g[i], 8), rank, i, steps=8)
    moe.moe_orthogonalize(g, out, _ws(n, rows, cols), steps=16)
    for i in (0, n - 1):
        assert torch.isfinite(out[i]).all()
        # 1.205 is the iteration's largest value on [0, 1.21]; bf16 rounds
        assert np.linalg.norm(out[i].double().cpu().numpy(), 2) <= 1.22
