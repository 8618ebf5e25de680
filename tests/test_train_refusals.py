"""A call of LayerTrain that is refused leaves the step before as it was: its
backward still gives that step's gradients."""
import os

import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from mixture_experts_layer_fp32_amd import _binding as B

T, D, E, K, I = 70, 64, 6, 2, 64


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not os.path.exists(B.LIB_PATH):  # build only when nothing is built yet
        from mixture_experts_layer_fp32_amd import build
        build.build()
    B.load_library()


def make(device, **kw):
    g = torch.Generator().manual_seed(3)
    w = [torch.randn(*s, generator=g) * 0.2 for s in ((E, D), (E, D, 2 * I), (E, I, D))]
    w = [w[0].to(device)] + [t.bfloat16().to(device) for t in w[1:]]
    return moe.LayerTrain(moe.make_desc(T=T, D=D, E=E, top_k=K, I=I), *w, device=device, **kw)


def rows(seed, device):
    return torch.randn(T, D, generator=torch.Generator().manual_seed(seed)).bfloat16().to(device)


@pytest.mark.parametrize("norm", [False, True])
def test_mask_without_balance_is_refused_first(norm):
    """Without a GPU: the refusal comes before any call."""
    lay = make("cpu", norm=norm)
    lay.x = kept = rows(0, "cpu")
    with pytest.raises(ValueError, match="mask: only with balance"):
        lay.forward(rows(1, "cpu"), mask=torch.ones(T, dtype=torch.bool))
    assert lay.x is kept


@pytest.mark.parametrize("kw", [dict(), dict(norm=True), dict(ckpt=True), dict(balance=0.1)],
                         ids=["plain", "norm", "ckpt", "balance"])
def test_backward_without_a_forward_is_refused(kw):
    """Without a GPU: it comes before any call. (The routing's positions would
    be whatever the memory held, and gradients are written through them.)"""
    with pytest.raises(RuntimeError, match="no forward"):
        make("cpu", **kw).backward(rows(2, "cpu"))


def test_scratch_of_another_device_is_refused():
    """(Some calls do not look where their tensors are.)"""
    pool = {}
    make("meta", ckpt=True, scratch=pool)
    with pytest.raises(ValueError, match="scratch: x_perm is on meta, the layer on cpu"):
        make("cpu", ckpt=True, scratch=pool)
    for t in [k for k in pool if not k.startswith("ws_")]:
        del pool[t]
    with pytest.raises(ValueError, match="scratch: ws_ffn is on meta"):
        make("cpu", ckpt=True, scratch=pool)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(norm=True), dict(ckpt=True, norm=True)],
                         ids=["plain", "norm", "ckpt"])
def test_refused_forward_leaves_the_step_before(kw):
    x, dout = rows(1, "cuda"), rows(2, "cuda")
    bad_x = [rows(4, "cuda").float(), rows(4, "cuda")[:-1], rows(4, "cuda")[:, ::2],
             rows(4, "cpu"), None]
    bad_mask = [torch.ones(T - 1, dtype=torch.uint8, device="cuda"),
                torch.ones(T, dtype=torch.int32, device="cuda"), torch.ones(T, dtype=torch.uint8),
                torch.ones(2 * T, dtype=torch.uint8, device="cuda")[::2]]
    for balance in (None, 0.1):
        lay = make("cuda", balance=balance, **kw)
        want = None
        for refuse in (False, True):
            lay.forward(x)
            if refuse:
                for b in bad_x:
                    with pytest.raises((ValueError, TypeError)):
                        lay.forward(b)
                for m in bad_mask:
                    with pytest.raises(ValueError, match="mask"):
                        lay.forward(rows(4, "cuda"), mask=m)
            lay.backward(dout)
            got = [t.clone() for t in (lay.dx, lay.dw_router, lay.dw_gate_up, lay.dw_down)]
            if want is None:
                want = got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
