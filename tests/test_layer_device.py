"""Layers whose tensors lie on another GPU than the current one run with theirs
current (shown without a GPU: what the calls would find is recorded)."""
import os

import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from mixture_experts_layer_fp32_amd import _binding as B
from mixture_experts_layer_fp32_amd import layer as L


class Out:
    """A tensor on GPU 1, as far as the layer asks."""
    dtype = torch.bfloat16

    def get_device(self):
        return 1


@pytest.fixture
def current(monkeypatch):
    """Current GPU 0; the GPU that is current at each call of the binding."""
    if not os.path.exists(B.LIB_PATH):  # build only when nothing is built yet
        from mixture_experts_layer_fp32_amd import build
        build.build()
    state, calls = [0], []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.was, state[0] = state[0], self.dev

        def __exit__(self, *_):
            state[0] = self.was

    class Recorder:
        """In place of the binding: records instead of calling."""
        def __getattr__(self, name):
            if name == "_current_device":
                return lambda: state[0]
            if name.startswith("moe_") and not name.endswith("_size"):
                return lambda *a, **kw: calls.append((name, state[0]))
            if name in ("_device_of", "_ptr_on", "_mask"):
                return lambda *a, **kw: 1
            return getattr(B, name)

    def use():
        monkeypatch.setattr(L, "B", Recorder())
        monkeypatch.setattr(torch.cuda, "device", Device)
    return use, calls, state


def weights(E=4, D=64, I=64):
    return torch.zeros(E, D), torch.zeros(E, D, 2 * I), torch.zeros(E, I, D)


def test_train_runs_on_its_own_gpu(current):
    use, calls, state = current
    w = [t if i == 0 else t.bfloat16() for i, t in enumerate(weights())]
    for kw in (dict(), dict(norm=True, ckpt=True, balance=0.1)):
        lay = moe.LayerTrain(moe.make_desc(T=8, D=64, E=4, top_k=2, I=64), *w, device="cpu", **kw)
        use()
        lay.out = Out()
        lay.forward(torch.zeros(8, 64, dtype=torch.bfloat16))
        lay.backward(torch.zeros(8, 64, dtype=torch.bfloat16))
    assert len(calls) > 10 and {dev for _, dev in calls} == {1}, calls
    assert state == [0]


def test_fp8_runs_on_its_own_gpu(current):
    use, calls, state = current
    u8 = torch.uint8
    gate_up = torch.zeros(4, 128, 64, dtype=u8), torch.zeros(4, 1, 1)
    down = torch.zeros(4, 64, 64, dtype=u8), torch.zeros(4, 1, 1)
    lay = moe.LayerForwardFP8(moe.make_desc(T=8, D=64, E=4, top_k=2, I=64), weights()[0], gate_up,
                              down, device="cpu")
    use()
    lay.out = Out()
    lay(torch.zeros(8, 64, dtype=torch.bfloat16))
    assert len(calls) >= 5 and {dev for _, dev in calls} == {1}, calls
    assert state == [0]
