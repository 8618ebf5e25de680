"""FP8 block products, 8-bit checkpoints and the balance loss without a GPU:
the oracles against torch's own E4M3 and against differences, and the calls
that are refused on the host before any HIP call."""
import ctypes
import os

import numpy as np
import pytest
import torch

from mixture_experts_layer_fp32_amd import _binding as B
from oracle import fp8_ckpt_balance_oracle as fo

P = ctypes.c_void_p(0x1000)   # never dereferenced: every call below fails its checks
ODD = ctypes.c_void_p(0x1008)


# Sizes whose launch would have 2^32 threads, and sizes past it.
@pytest.mark.parametrize("rows,K", [(2 ** 28 - 15, 64), (2 ** 28 - 1, 64), (2 ** 28, 64),
                                    (2 ** 27 - 1, 128)])
def test_sizes_past_a_launch(lib, rows, K):
    assert lib.moe_fp8_quantize_rows(rows, K, B.MOE_BF16, P, P, P, None) == B.MOE_ERR_UNSUPPORTED
    assert lib.moe_ckpt_save_rows(rows, K, B.MOE_BF16, P, P, P, None) == B.MOE_ERR_UNSUPPORTED
    T = min(2 ** 31 - 1, rows * 8)
    assert lib.moe_router_backward_dense(T, 8, K, B.MOE_BF16, P, P, P, 0, P, None,
                                         None, 0, None) == B.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):  # build only when nothing is built yet
        from mixture_experts_layer_fp32_amd import build
        build.build()
    return B.load_library()


def desc(**kw):
    return B.make_desc(**{**dict(T=64, D=256, E=8, top_k=2, I=192), **kw})


# ---- the oracles ----
def test_e4m3_encode_matches_torch():
    g = np.random.default_rng(0)
    v = np.concatenate([g.uniform(-448, 448, 4000), g.normal(size=4000) * 2.0 ** -7,
                        fo.E4M3, -fo.E4M3, fo._MID, -fo._MID, [0.0, -0.0]]).astype(np.float32)
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fo.e4m3_encode(v), ref)
    assert np.array_equal(fo.e4m3_decode(ref),
                          torch.from_numpy(ref).view(torch.float8_e4m3fn).double().numpy())


def test_fp8_rows_error_is_half_a_step():
    g = np.random.default_rng(1)
    x = (g.normal(size=(9, 320)) * np.exp(g.normal(size=(9, 1)))).astype(np.float32)
    codes, scales = fo.fp8_rows(x)
    y = fo.fp8_row_values(codes, scales)
    s = np.repeat(scales.T, 128, 1)[:, :320]
    # half an E4M3 step (2^-4 of the value, 2^-10 of the scale when subnormal)
    # and the roundings of 1/s and of the product (2^-23)
    assert (np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) * 1.00001
            + 2.0 ** -22 * np.abs(x)).all()


def test_ckpt_error_is_half_a_step():
    g = np.random.default_rng(2)
    x = (g.normal(size=(9, 320)) * np.exp(3 * g.normal(size=(9, 1)))).astype(np.float32)
    codes, bits = fo.ckpt_rows(x)
    s = np.repeat(fo.bf16_values(bits), 32, 1)
    # half a step, and the fp32 roundings of 1/s and of the product (127 steps
    # of 2^-24 each)
    assert (np.abs(fo.ckpt_values(codes, bits) - x) <= (0.5 + 127 * 2.0 ** -23) * s).all()
    top = np.abs(x.reshape(9, -1, 32)).max(2)
    assert (fo.bf16_values(bits) * 127 >= top * (1 - 2.0 ** -22)).all()
    assert (fo.bf16_values(bits) * 127 <= top * (1 + 2.0 ** -7)).all()


def test_ckpt_of_the_largest_values_is_finite():
    top = np.finfo(np.float32).max
    m = np.array([top, -top, 255 * 2.0 ** 120, 127 * 2.0 ** 121, 126.4 * 2.0 ** 121, 2.0 ** 127])
    x = np.concatenate([np.diag(m), np.outer(m, np.linspace(-1, 1, 26))], 1).astype(np.float32)
    codes, bits = fo.ckpt_rows(x)
    back = fo.ckpt_values(codes, bits)
    s = np.repeat(fo.bf16_values(bits), 32, 1)
    # half a step, and 1/128 of up to 128 steps with the largest scale
    assert (np.abs(back.astype(np.float64) - x) <= 1.5 * (1 + 2.0 ** -16) * s).all()
    assert torch.isfinite(torch.from_numpy(back).to(torch.bfloat16)).all()


def test_balance_gradient_against_differences():
    g = np.random.default_rng(3)
    T, E, k, coef = 6, 5, 2, 0.3
    z = g.normal(size=(T, E))
    topk = np.argsort(-z, 1)[:, :k].astype(np.int32)
    mask = np.array([1, 1, 0, 1, 1, 0], np.uint8)
    counts, N, _, _ = fo.balance_loss(z, topk, coef, mask)
    d = fo.balance_backward(z, coef, k, counts, N, 1.7, mask)
    h = 1e-5
    for t, e in np.ndindex(T, E):
        dz = np.zeros_like(z)
        dz[t, e] = h
        num = 1.7 * (fo.balance_loss(z + dz, topk, coef, mask)[3]
                     - fo.balance_loss(z - dz, topk, coef, mask)[3]) / (2 * h)
        assert abs(num - d[t, e]) <= 1e-9


def test_balance_loss_of_an_even_load_is_its_coefficient():
    E, k = 4, 2
    topk = np.array([[0, 1], [2, 3]] * 3, np.int32)
    assert abs(fo.balance_loss(np.zeros((6, E)), topk, 0.25)[3] - 0.25) < 1e-12
    # everything on two experts that the router is sure of: E / k times that
    z = np.where(np.arange(E) < 2, 0.0, -60.0)[None].repeat(6, 0)
    topk = np.array([[0, 1]] * 6, np.int32)
    assert abs(fo.balance_loss(z, topk, 0.25)[3] - 0.25 * E / k) < 1e-12


# ---- refusals ----
INV, UNS, WS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("args,want", [
    ((-1, 128, 1, P, P, P), INV), ((4, 0, 1, P, P, P), INV), ((4, 96, 1, P, P, P), INV),
    ((4, 128, 2, P, P, P), UNS), ((4, 128, 7, P, P, P), UNS), ((4, 262208, 1, P, P, P), UNS),
    ((2 ** 31, 64, 1, P, P, P), UNS), ((2 ** 17, 2 ** 17, 1, P, P, P), UNS),
    ((4, 128, 1, None, P, P), INV), ((4, 128, 1, P, None, P), INV), ((4, 128, 1, P, P, None), INV),
    ((4, 128, 1, ODD, P, P), INV), ((4, 128, 1, P, ODD, P), INV),
    ((0, 128, 1, None, None, None), 0),
])
def test_fp8_quantize_rows_refusals(lib, args, want):
    assert lib.moe_fp8_quantize_rows(*args, None) == want


@pytest.mark.parametrize("args,want", [
    ((-1, 64, 64, 1, P, P, P), INV), ((1, 32, 64, 1, P, P, P), INV), ((1, 64, 0, 1, P, P, P), INV),
    ((1, 64, 100, 1, P, P, P), INV), ((1, 64, 64, 2, P, P, P), UNS),
    ((1025, 64, 64, 1, P, P, P), UNS), ((1, 524352, 64, 1, P, P, P), UNS),
    ((1024, 524288, 524288, 1, P, P, P), UNS), ((1, 64, 64, 1, None, P, P), INV),
    ((1, 64, 64, 1, ODD, P, P), INV), ((0, 64, 64, 1, None, None, None), 0),
])
def test_fp8_pack_weights_refusals(lib, args, want):
    assert lib.moe_fp8_pack_weights(*args, None) == want


def test_fp8_product_refusals(lib):
    up, down, ffn = lib.moe_expert_gate_up_fp8, lib.moe_expert_down_fp8, lib.moe_expert_ffn_fp8
    d = desc()
    r = ctypes.byref(d)
    for f in (up, down):
        ok = [1, 192, 10, P, P, P, P, P, P]
        for i, v, want in ((0, 0, INV), (0, 1025, UNS), (1, 0, INV), (1, 100, UNS), (2, -1, INV),
                           (2, 2 ** 31, UNS), (3, None, INV), (4, None, INV), (6, None, INV),
                           (7, None, INV), (8, None, INV), (3, ODD, INV), (6, ODD, INV),
                           (8, ODD, INV)):
            a = list(ok)
            a[i] = v
            assert f(r, *a, None) == want, (i, v)
        assert f(r, 2, 192, 10, P, P, None, P, P, P, None) == INV  # no offsets: one expert
        assert f(r, 1, 192, 0, None, None, None, None, None, None, None) == 0
        assert f(None, *ok, None) == INV
        assert f(ctypes.byref(desc(dtype="f32")), *ok, None) == UNS
        big = desc(D=262144)
        assert f(ctypes.byref(big), 1, 1024, 10, P, P, P, P, P, P, None) == UNS
    need = lib.moe_ffn_fp8_workspace_size(r, 192, 10)
    assert need >= 10 * 192 * 3 + 2 * 10 * 4
    assert ffn(r, 1, 192, 10, P, P, P, P, P, P, P, P, P, need - 1, None) == WS
    assert ffn(r, 1, 192, 10, P, P, P, P, P, P, P, P, None, need, None) == INV
    assert ffn(r, 1, 192, 10, P, P, P, P, P, P, P, P, ODD, need, None) == INV
    assert lib.moe_ffn_fp8_workspace_size(r, 100, 10) == 0
    assert lib.moe_ffn_fp8_workspace_size(r, 192, -1) == 0


@pytest.mark.parametrize("args,want", [
    ((-1, 64, 1, P, P, P), INV), ((4, 16, 1, P, P, P), INV), ((4, 64, 2, P, P, P), UNS),
    ((4, 524320, 1, P, P, P), UNS), ((4, 64, 1, None, P, P), INV), ((4, 64, 1, P, P, None), INV),
    ((4, 64, 1, ODD, P, P), INV), ((4, 64, 1, P, ODD, P), INV),
    ((0, 64, 1, None, None, None), 0),
])
def test_ckpt_save_refusals(lib, args, want):
    assert lib.moe_ckpt_save_rows(*args, None) == want


@pytest.mark.parametrize("args,want", [
    ((-1, 4, 64, 1, P, P, P, P), INV), ((4, -1, 64, 1, P, P, P, P), INV),
    ((4, 4, 48, 1, P, P, P, P), INV), ((5, 4, 64, 1, P, P, None, P), INV),
    ((4, 4, 64, 2, P, P, P, P), UNS), ((4, 4, 64, 1, None, P, P, P), INV),
    ((4, 4, 64, 1, P, None, P, P), INV), ((4, 4, 64, 1, P, P, P, None), INV),
    ((4, 4, 64, 1, ODD, P, P, P), INV), ((4, 4, 64, 1, P, P, P, ODD), INV),
    ((0, 4, 64, 1, None, None, None, None), 0), ((4, 0, 64, 1, None, None, P, None), 0),
])
def test_ckpt_restore_refusals(lib, args, want):
    assert lib.moe_ckpt_restore_rows(*args, None) == want


def test_ckpt_ffn_refusals(lib):
    d = desc()
    r = ctypes.byref(d)
    up, bwd = lib.moe_expert_gate_up_train_ckpt, lib.moe_expert_gate_up_backward_ckpt
    full, fbwd = lib.moe_expert_ffn_train_ckpt, lib.moe_expert_ffn_backward_ckpt
    a = [1, 192, 10, P, P, P, P, P, P]
    for i in (3, 5, 6, 7, 8):
        b = list(a)
        b[i] = None
        assert up(r, *b, None) == INV, i
    assert up(r, *a[:7], ODD, P, None) == INV
    b = [1, 192, 10, P, P, P, P, P, P, P]
    for i in (3, 5, 6, 7, 8, 9):
        c = list(b)
        c[i] = None
        assert bwd(r, *c, None) == INV, i
    for f, args in ((up, a), (bwd, b)):
        assert f(ctypes.byref(desc(dtype="f32")), *args, None) == UNS
        assert f(ctypes.byref(desc(packed=True)), *args, None) == UNS
        assert f(ctypes.byref(desc(y_fp16=True)), *args, None) == UNS
        two = [2] + args[1:4] + [None] + args[5:]
        assert f(r, *two, None) == INV
    assert bwd(ctypes.byref(desc(norm_topk=False)), *b, None) == UNS
    need = B.moe_ffn_workspace_size(d, 192, 10)
    assert full(r, 1, 192, 10, P, P, P, P, P, P, P, P, need - 1, None) == WS
    need = B.moe_ffn_backward_workspace_size(d, 192, 10)
    assert fbwd(r, 1, 192, 10, P, P, P, P, P, P, P, P, P, P, P, need - 1, None) == WS
    assert fbwd(r, 1, 192, 10, P, P, P, P, P, ODD, P, P, P, P, P, need, None) == INV


def test_balance_refusals(lib):
    f = lib.moe_balance_loss
    need = lib.moe_balance_loss_workspace_size(64, 8)
    ok = [64, 8, 2, 0, P, P, None, 0.1, P, P, P, P, P, need]
    for i, v, want in ((0, -1, INV), (1, 0, INV), (2, 0, INV), (2, 9, INV), (3, 3, UNS),
                       (4, None, INV), (5, None, INV), (7, float("inf"), INV),
                       (7, float("nan"), INV), (8, None, INV), (9, None, INV), (10, None, INV),
                       (11, None, INV), (12, None, INV), (13, need - 1, WS)):
        a = list(ok)
        a[i] = v
        assert f(*a, None) == want, (i, v)
    assert f(*([64, 1025] + ok[2:]), None) == UNS
    assert f(*([64, 32, 17] + ok[3:]), None) == UNS
    assert lib.moe_balance_loss_workspace_size(-1, 8) == 0
    assert lib.moe_balance_loss_workspace_size(64, 1025) == 0
    g = lib.moe_balance_loss_backward
    ok = [64, 8, 2, 0, P, P, None, 0.1, P, P, None, P, P]
    for i, v in ((4, None), (5, None), (8, None), (9, None), (12, None)):
        a = list(ok)
        a[i] = v
        assert g(*a, None) == INV, i
    assert g(0, 8, 2, 0, None, None, None, 0.1, None, None, None, None, None, None) == 0


def test_router_dense_refusals(lib):
    f = lib.moe_router_backward_dense
    T, E, D = 4096, 8, 256
    need = lib.moe_router_backward_dense_workspace_size(T, E, D)
    ok = [T, E, D, 0, P, P, P, 0, P, P, P, max(need, 1)]
    for i, v, want in ((0, -1, INV), (1, 0, INV), (2, 100, INV), (2, 0, INV), (3, 2, UNS),
                       (4, None, INV), (5, None, INV), (6, None, INV), (7, 2, INV), (5, ODD, INV),
                       (6, ODD, INV), (8, ODD, INV), (9, ODD, INV), (10, ODD, INV),
                       (1, 1025, UNS), (2, 262208, UNS)):
        a = list(ok)
        a[i] = v
        assert f(*a, None) == want, (i, v)
    if need:
        assert f(*ok[:11], need - 1, None) == WS
        assert f(*ok[:10], None, need, None) == WS
    assert f(2 ** 31 - 1, E, 262144, 0, P, P, P, 0, P, None, None, 0, None) == UNS
    assert lib.moe_router_backward_dense_workspace_size(-1, E, D) == 0


def test_binding_names_what_is_wrong():
    with pytest.raises(ValueError, match="x: must be a GPU tensor"):
        B.moe_fp8_quantize_rows(torch.zeros(2, 128), None, None)
    with pytest.raises(ValueError, match=r"x: expected \[rows, D\]"):
        B.moe_ckpt_save_rows(torch.zeros(128), None, None)
    with pytest.raises(ValueError, match="w: expected"):
        B.moe_fp8_pack_weights(torch.zeros(2, 128), None, None)
    with pytest.raises(ValueError, match="logits: dtype"):
        B.moe_balance_loss(torch.zeros(2, 8, dtype=torch.float64), None, 0.1, None, None, None,
                           None, None)
    with pytest.raises(ValueError, match="out: rows of 64, codes of 128"):
        B.moe_ckpt_restore_rows(torch.zeros(2, 128, dtype=torch.int8), None, torch.zeros(2, 64))
