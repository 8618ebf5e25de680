"""Layer norm and the Muon update without a GPU: the oracle's gradient against
differences, what the oracle's iteration does, and the calls that are refused
on the host before any HIP call."""
import ctypes
import os

import numpy as np
import pytest
import torch

from mixture_experts_layer_fp32_amd import _binding as B
from oracle import norm_update_oracle as ou

CPU = torch.zeros(1).get_device()
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails its checks


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):  # build only when nothing is built yet
        from mixture_experts_layer_fp32_amd import build
        build.build()
    return B.load_library()


def test_layer_norm_gradient_against_differences():
    g = np.random.default_rng(0)
    x, dy = g.normal(size=(3, 7)), g.normal(size=(3, 7))
    gamma, beta = g.normal(size=7), g.normal(size=7)

    def loss(x, gamma, beta):
        return (ou.layer_norm(x, gamma, beta)[0] * dy).sum()

    _, mean, rstd = ou.layer_norm(x, gamma, beta)
    dx, dgamma, dbeta = ou.layer_norm_backward(x, dy, gamma, mean, rstd)
    step = 1e-5
    for i in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[i] = step
        d = (loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * step)
        assert abs(d - dx[i]) <= 1e-8 * (1 + abs(d))  # second differences: O(step^2)
    for j in range(7):
        e = np.zeros(7)
        e[j] = step
        d = (loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * step)
        assert abs(d - dgamma[j]) <= 1e-8 * (1 + abs(d))
        d = (loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * step)
        assert abs(d - dbeta[j]) <= 1e-8 * (1 + abs(d))


def test_iteration_maps_singular_values_by_the_quintic():
    g = np.random.default_rng(1)
    w = g.normal(size=(6, 11))
    u, s, vt = np.linalg.svd(w, full_matrices=False)
    a, b, c = ou.COEFS
    t = s / (np.linalg.norm(w) + 1e-7)
    for _ in range(5):
        t = a * t + b * t ** 3 + c * t ** 5
    assert np.abs(ou.orthogonalize(w) - (u * t) @ vt).max() < 1e-12
    assert np.abs(ou.orthogonalize(w.T) - ou.orthogonalize(w).T).max() < 1e-12


def test_layer_norm_refusals(lib):
    def fwd(rows=4, D=8, dtype=B.MOE_BF16, x=FAKE, eps=1e-5, y=FAKE):
        return lib.moe_layer_norm(rows, D, dtype, x, FAKE, FAKE, eps, y, None, None, None)

    assert fwd(rows=-1) == B.MOE_ERR_INVALID_ARG
    assert fwd(D=0) == B.MOE_ERR_INVALID_ARG
    assert fwd(D=B.MOE_MAX_WIDTH + 1) == B.MOE_ERR_UNSUPPORTED
    assert fwd(rows=1 << 39) == B.MOE_ERR_UNSUPPORTED
    assert fwd(dtype=B.MOE_F16) == B.MOE_ERR_UNSUPPORTED
    assert fwd(eps=-1e-5) == B.MOE_ERR_INVALID_ARG
    assert fwd(eps=float("nan")) == B.MOE_ERR_INVALID_ARG
    assert fwd(eps=float("inf")) == B.MOE_ERR_INVALID_ARG
    assert fwd(x=None) == B.MOE_ERR_INVALID_ARG
    assert fwd(y=None) == B.MOE_ERR_INVALID_ARG
    assert fwd(rows=0, x=None, y=None) == B.MOE_OK  # nothing to do

    need = lib.moe_layer_norm_backward_workspace_size(4, 8)
    assert need > 0
    assert lib.moe_layer_norm_backward_workspace_size(-1, 8) == 0
    assert lib.moe_layer_norm_backward_workspace_size(4, 0) == 0

    def bwd(rows=4, D=8, dtype=B.MOE_F32, x=FAKE, dy=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE,
            dgamma=FAKE, ws=FAKE, n=need):
        return lib.moe_layer_norm_backward(rows, D, dtype, x, dy, None, mean, rstd, None, dx,
                                           dgamma, None, ws, n, None)

    assert bwd(rows=-1) == B.MOE_ERR_INVALID_ARG
    assert bwd(dtype=9) == B.MOE_ERR_UNSUPPORTED
    for name in ("x", "dy", "mean", "rstd", "dx", "ws"):
        assert bwd(**{name: None}) == B.MOE_ERR_INVALID_ARG, name
    assert bwd(n=need - 1) == B.MOE_ERR_WORKSPACE
    assert bwd(rows=0, x=None, dy=None, mean=None, rstd=None, dx=None, dgamma=None, ws=None,
               n=0) == B.MOE_OK


def _mats(data=0x1000, dtype=B.MOE_F32, ld=16, stride=128):
    return B.moe_matrices(data, dtype, ld, stride)


def test_orthogonalize_refusals(lib):
    need = lib.moe_orthogonalize_workspace_size(2, 8, 16, 5)
    assert need > 0

    def call(n=2, rows=8, cols=16, g=_mats(), steps=5, eps=1e-7, out=_mats(0x9000), ws=0x10000,
             size=need):
        return lib.moe_orthogonalize(n, rows, cols, ctypes.byref(g) if g else None, steps, eps,
                                     ctypes.byref(out) if out else None,
                                     ctypes.c_void_p(ws) if ws else None, size, None)

    assert call(n=-1) == B.MOE_ERR_INVALID_ARG
    assert call(rows=0) == B.MOE_ERR_INVALID_ARG
    assert call(cols=0) == B.MOE_ERR_INVALID_ARG
    assert call(steps=0) == B.MOE_ERR_INVALID_ARG
    assert call(steps=17) == B.MOE_ERR_INVALID_ARG
    assert call(eps=-1.0) == B.MOE_ERR_INVALID_ARG
    assert call(eps=float("nan")) == B.MOE_ERR_INVALID_ARG
    assert call(n=65536) == B.MOE_ERR_UNSUPPORTED
    assert call(rows=B.MOE_MAX_WIDTH + 1) == B.MOE_ERR_UNSUPPORTED
    assert call(rows=32769, cols=32769) == B.MOE_ERR_UNSUPPORTED
    assert call(n=2048, rows=4096, cols=4096) == B.MOE_ERR_UNSUPPORTED  # 2^23 tiles of 64 x 64
    for bad, code in ((_mats(data=None), B.MOE_ERR_INVALID_ARG),
                      (_mats(ld=15), B.MOE_ERR_INVALID_ARG),
                      (_mats(stride=15), B.MOE_ERR_INVALID_ARG),
                      (_mats(stride=-128), B.MOE_ERR_INVALID_ARG),
                      (_mats(dtype=B.MOE_F16), B.MOE_ERR_UNSUPPORTED),
                      (_mats(ld=1 << 41), B.MOE_ERR_UNSUPPORTED), (None, B.MOE_ERR_INVALID_ARG)):
        assert call(g=bad) == code
        assert call(out=bad) == code
    assert call(ws=None) == B.MOE_ERR_INVALID_ARG
    assert call(ws=0x10010) == B.MOE_ERR_INVALID_ARG  # misaligned
    assert call(size=need - 1) == B.MOE_ERR_WORKSPACE
    assert call(n=0, g=None, out=None, ws=None, size=0) == B.MOE_OK
    assert lib.moe_orthogonalize_workspace_size(2, 0, 16, 5) == 0
    assert lib.moe_orthogonalize_workspace_size(0, 8, 16, 5) == 0


def test_muon_update_refusals(lib):
    need = lib.moe_orthogonalize_workspace_size(2, 8, 16, 5)
    good = dict(lr=0.1, mu=0.9, weight_decay=0.0, scale=1.0, eps=1e-7, nesterov=1, steps=5)

    def call(m=_mats(0x5000), w=_mats(0x9000), g=_mats(), size=need, desc=True, **kw):
        d = B.moe_muon_desc(**{**good, **kw})
        return lib.moe_muon_update(2, 8, 16, ctypes.byref(d) if desc else None, ctypes.byref(g),
                                   ctypes.byref(m), ctypes.byref(w), ctypes.c_void_p(0x10000),
                                   size, None)

    for name in ("lr", "mu", "weight_decay", "scale", "eps"):
        assert call(**{name: float("nan")}) == B.MOE_ERR_INVALID_ARG, name
        assert call(**{name: float("inf")}) == B.MOE_ERR_INVALID_ARG, name
    assert call(eps=-1.0) == B.MOE_ERR_INVALID_ARG
    assert call(nesterov=2) == B.MOE_ERR_INVALID_ARG
    assert call(steps=0) == B.MOE_ERR_INVALID_ARG
    assert call(desc=False) == B.MOE_ERR_INVALID_ARG
    assert call(m=_mats(0x5000, dtype=B.MOE_BF16)) == B.MOE_ERR_UNSUPPORTED
    assert call(w=_mats(0x9000, dtype=7)) == B.MOE_ERR_UNSUPPORTED
    assert call(g=_mats(ld=3)) == B.MOE_ERR_INVALID_ARG
    assert call(size=need - 1) == B.MOE_ERR_WORKSPACE


def test_binding_refuses_host_tensors_and_shapes(lib):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        B.moe_layer_norm(x, None, None, 1e-5, x)
    with pytest.raises(ValueError):
        B.moe_layer_norm(torch.zeros(8), None, None, 1e-5, x)
    with pytest.raises(ValueError):
        B.moe_orthogonalize(x, x, torch.zeros(4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B._matrices(CPU, torch.zeros(2, 4, 8).transpose(1, 2), "g")  # columns not adjacent
    with pytest.raises(ValueError):
        B._matrices(CPU, torch.zeros(2, 4, 8, dtype=torch.float16), "g")
    with pytest.raises(ValueError):
        B._matrices(CPU, torch.zeros(8), "g")
    m = B._matrices(CPU, torch.zeros(3, 4, 16)[:, :, :8], "g")
    assert (m.ld, m.stride) == (16, 64)
