"""The bytes that a LayerTrain keeps from its forward to its backward (counted
on CPU tensors: the layer allocates the same on a GPU)."""
import os

import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from mixture_experts_layer_fp32_amd import _binding as B


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not os.path.exists(B.LIB_PATH):  # build only when nothing is built yet
        from mixture_experts_layer_fp32_amd import build
        build.build()
    B.load_library()


def make(T, D, E, k, I, Is, **kw):
    bf = torch.bfloat16
    shared = dict(shared_gate_up=torch.empty(D, 2 * Is, dtype=bf),
                  shared_down=torch.empty(Is, D, dtype=bf)) if Is else {}
    return moe.LayerTrain(moe.make_desc(T=T, D=D, E=E, top_k=k, I=I, I_shared=Is),
                          torch.empty(E, D), torch.empty(E, D, 2 * I, dtype=bf),
                          torch.empty(E, I, D, dtype=bf), device="cpu", **shared, **kw)


def tensors(lay):
    """{address: bytes} of the layer's tensors, weights' gradients left out."""
    return {t.data_ptr(): t.numel() * t.element_size() for name, t in vars(lay).items()
            if isinstance(t, torch.Tensor) and t.numel() and not name.startswith(("dw_", "dnorm"))}


SIZES = [(1024, 512, 8, 2, 1024, 256), (512, 256, 16, 4, 256, 0), (640, 320, 6, 2, 192, 64)]


@pytest.mark.parametrize("T,D,E,k,I,Is", SIZES)
@pytest.mark.parametrize("norm", [False, True])
def test_a_quarter_of_the_bytes_with_a_shared_scratch(T, D, E, k, I, Is, norm):
    pool = {}
    plain = make(T, D, E, k, I, Is, norm=norm)
    kept = make(T, D, E, k, I, Is, norm=norm, ckpt=True, scratch=pool)
    # what the plain step keeps: bf16 x_perm, fp32 y_perm and G | U
    before = T * k * (2 * D + 4 * D + 8 * I) + T * 8 * Is
    assert before == sum(t.numel() * t.element_size()
                         for t in (plain.x_perm, plain.y_perm, plain.gu, plain.gu_sh)
                         if t is not None)
    # in 8.5 bits: x once a token, y, G | U
    after = (T * (D + 2 * Is) + T * k * (D + 2 * I)) * 17 // 16
    own = tensors(kept)
    for t in pool.values():
        own.pop(t.data_ptr(), None)
    # with it the layer's own output, dx, and what the routing left
    rest = 2 * T * D * 2 + T * k * 16 + T * 8 + E * 8 + kept.ws_route.numel() + kept.ws_perm.numel()
    assert after <= sum(own.values()) <= after + rest + 4096
    assert after <= 0.3 * before
    # a second layer adds its own bytes and no others
    make(T, D, E, k, I, Is, norm=norm, ckpt=True, scratch=pool)
    assert {t.data_ptr() for t in pool.values()} <= set(tensors(kept))


@pytest.mark.parametrize("T,D,E,k,I,Is", SIZES)
def test_without_a_scratch_the_layer_holds_x_perm_and_y_perm_too(T, D, E, k, I, Is):
    kept = make(T, D, E, k, I, Is, ckpt=True)
    own = tensors(kept)
    for t in (kept.x_perm, kept.y_perm, kept.gu_q, kept.x_q, kept.y_q):
        assert t.data_ptr() in own
