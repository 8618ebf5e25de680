"""The stream that the short calls are enqueued on: torch's current one, however
the binding asks for it."""
import importlib.util

import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from mixture_experts_layer_fp32_amd import _binding as B


def test_public_interface_where_torch_has_no_other(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("binding_without", B.__file__)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod._current_stream is mod._public_stream


@pytest.mark.gpu
@pytest.mark.parametrize("ask", ["_current_stream", "_public_stream"])
def test_calls_run_on_the_current_stream(ask, monkeypatch):
    monkeypatch.setattr(B, "_current_stream", getattr(B, ask))
    x = torch.randn(64, 96, device="cuda")
    ref = torch.empty_like(x)
    moe.moe_layer_norm(x, None, None, 1e-5, ref)
    torch.cuda.synchronize()
    for s in (torch.cuda.default_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert B._current_stream(0) == s.cuda_stream
            y = torch.zeros_like(x)
            moe.moe_layer_norm(x, None, None, 1e-5, y)
            s.synchronize()
            assert torch.equal(y, ref)
