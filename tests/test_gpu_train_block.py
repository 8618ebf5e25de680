"""A training step of the pre-norm block on the GPU: LayerTrain with its norm,
forward and backward, then ExpertMuon; each part against the float64 oracles on
what the parts before it left, and the whole step captured into a graph."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
import workloads as wl
from oracle import moe_backward_oracle as ob
from oracle import norm_update_oracle as ou
from parity import npi, np32, to_dev
from test_gpu_orth import HALF, TOL, U

pytestmark = pytest.mark.gpu

BLOCKS = {
    "bf16_shared": wl.Workload("block_bf16", T=200, D=128, E=8, k=2, I=192, I_shared=64),
    "bf16": wl.Workload("block_bf16_plain", T=333, D=192, E=12, k=3, I=64),
    "f32": wl.Workload("block_f32", T=97, D=64, E=6, k=2, I=128, dtype="f32", I_shared=64),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


def _block(w, seed=3):
    g = torch.Generator().manual_seed(seed)
    inp = wl.make_inputs(w, seed=seed)
    for k in ("w_gate_up", "w_down", "shared_gate_up", "shared_down"):
        if inp[k] is not None:
            inp[k] = (inp[k].float() * 5).to(inp[k].dtype)
    inp["x"] = (inp["x"].float() * 2 + 0.5 * torch.randn(w.D, generator=g)).to(w.torch_dtype)
    dv = to_dev(inp)
    gamma = (1 + 0.2 * torch.randn(w.D, generator=g)).cuda()
    beta = (0.1 * torch.randn(w.D, generator=g)).cuda()
    d = moe.make_desc(T=w.T, D=w.D, E=w.E, top_k=w.k, I=w.I, I_shared=w.I_shared, dtype=w.dtype)
    lay = moe.LayerTrain(d, dv["w_router"], dv["w_gate_up"], dv["w_down"],
                         shared_gate_up=dv["shared_gate_up"], shared_down=dv["shared_down"],
                         norm=True, norm_gamma=gamma, norm_beta=beta)
    dout = torch.randn(w.T, w.D, generator=g).to(w.torch_dtype).cuda()
    return lay, dv, dout, gamma, beta


@pytest.mark.parametrize("name", sorted(BLOCKS))
def test_training_step(name):
    w = BLOCKS[name]
    lay, dv, dout, gamma, beta = _block(w)
    lay.forward(dv["x"])
    lay.backward(dout)
    torch.cuda.synchronize()
    x, f32 = np32(dv["x"]).astype(np.float64), w.dtype == "f32"
    # The norm in front: a row of at most 192 values of size up to 10.
    h, mean, rstd = ou.layer_norm(x, np32(gamma), np32(beta))
    assert np.all(np.abs(np32(lay.h) - h) <= HALF[w.torch_dtype] * np.abs(h) + 1e-5)
    # The layer without a norm, on h, gives the same routing and the same sum
    # of the experts: out - x = out' - h, to the two outputs' roundings.
    d = lay.d
    plain = moe.LayerTrain(d, dv["w_router"], dv["w_gate_up"], dv["w_down"],
                           shared_gate_up=dv["shared_gate_up"], shared_down=dv["shared_down"])
    out = np32(plain.forward(lay.h))
    torch.cuda.synchronize()
    assert torch.equal(plain.topk_idx, lay.topk_idx) and torch.equal(plain.y_perm, lay.y_perm)
    got = np32(lay.out)
    assert np.all(np.abs((got - x) - (out - np32(lay.h)))
                  <= 2 * HALF[w.torch_dtype] * (np.abs(got) + np.abs(out)) + 1e-5)
    # Its backward has the same weight gradients, bit for bit.
    plain.backward(dout)
    torch.cuda.synchronize()
    names = ["dw_router", "dw_gate_up", "dw_down"]
    names += ["dw_shared_gate_up", "dw_shared_down"] if w.I_shared else []
    for k in names:
        assert torch.equal(getattr(plain, k), getattr(lay, k)), k
    # dh: the layer's input gradient without the residual.
    layer = ob.layer_backward(np32(lay.h), np32(dv["w_router"]), np32(dv["w_gate_up"]),
                              np32(dv["w_down"]), w.k, np32(dout),
                              shared_gate_up=np32(dv["shared_gate_up"]),
                              shared_down=np32(dv["shared_down"]),
                              routing=(npi(lay.topk_idx), np32(lay.topk_w)))
    dh = layer["dx"] - np32(dout)
    err = np.linalg.norm(np32(lay.dh) - dh) / np.linalg.norm(dh)
    assert err < (1e-4 if f32 else 1e-2), err  # the layer's own backward tolerances
    # Back through the norm, from the dh that it was given.
    rdx, rdg, rdb = ou.layer_norm_backward(x, np32(lay.dh), np32(gamma), np32(lay.mean),
                                           np32(lay.rstd), np32(dout))
    assert np.all(np.abs(np32(lay.dx) - rdx) <= HALF[w.torch_dtype] * np.abs(rdx) + 1e-4
                  * np.abs(rdx).max())
    a = np.abs(np32(lay.dh)).sum(0)
    assert np.all(np.abs(np32(lay.dnorm_beta) - rdb) <= (w.T + 40) * U * a)
    assert np.all(np.abs(np32(lay.dnorm_gamma) - rdg) <= (w.T + 40) * U * 12 * a)
    # The Muon step, twice (the second with momentum), from the gradients as
    # they are.
    opt = moe.ExpertMuon(lay, weight_decay=0.1)
    lr = 0.02
    for _ in range(2):
        before = {k: (np32(lay.w[k]).astype(np.float64), np32(m).astype(np.float64))
                  for k, m in opt.momentum.items()}
        opt.step(lr)
        torch.cuda.synchronize()
        for k, (w0, m0) in before.items():
            g = np32(getattr(lay, "d" + k if k.startswith("w_") else "dw_" + k))
            w1, m1, w0, m0, g = (t.reshape(-1, *t.shape[-2:]) for t in
                                 (np32(lay.w[k]), np32(opt.momentum[k]), w0, m0, g))
            cols = w0.shape[2] // 2 if "gate_up" in k else w0.shape[2]
            for e in range(w0.shape[0]):
                for c in range(0, w0.shape[2], cols):
                    s = (e, slice(None), slice(c, c + cols))
                    scale = 0.2 * max(w0.shape[1], cols) ** 0.5
                    rm, rw = ou.muon_update(g[s], m0[s], w0[s], lr, weight_decay=0.1, scale=scale)
                    assert np.all(np.abs(m1[s] - rm) <= 3 * U * (np.abs(g[s]) + np.abs(m0[s])))
                    excess = np.maximum(np.abs(w1[s] - rw) - (HALF[w.torch_dtype] + U) * np.abs(rw)
                                        - 4 * U * np.abs(w0[s]), 0.0)
                    assert np.linalg.norm(excess) <= lr * scale * (TOL + 4 * U * 8), (k, e, c)


def test_block_gradient_against_differences():
    """dx of the whole fp32 block along random directions v (64 values, norm
    about 8) against differences of the block's own forward, step 1e-2: a
    change of 0.08 in a row of norm 16. Rounding: outputs of size 4 with
    relative errors of 1e-6, summed over 64 and divided by 2e-2, 2e-3; the
    third derivative: (0.08 / 16)^2 = 2.5e-5 of the gradient, times the
    layer's own curvature, 100 at most for weights five times the usual.
    Together well below 0.05 of the row's gradient norm (about 8)."""
    w = BLOCKS["f32"]
    lay, dv, dout, _, _ = _block(w)
    x = dv["x"]
    lay.forward(x)
    lay.backward(dout)
    dx, idx = lay.dx.double(), lay.topk_idx.clone()
    g = torch.Generator().manual_seed(9)
    step, checked = 1e-2, 0
    for _ in range(8):
        v = torch.randn(w.T, w.D, generator=g).cuda()
        up = lay.forward(x + step * v).double().clone()
        same = (lay.topk_idx == idx).all(1)
        down = lay.forward(x - step * v).double().clone()
        same &= (lay.topk_idx == idx).all(1)  # the choice of experts has no gradient
        diff = ((up - down) * dout.double()).sum(1) / (2 * step)
        want = (dx * v.double()).sum(1)
        assert torch.all(((diff - want).abs() <= 0.05 * dx.norm(dim=1))[same])
        checked += int(same.sum())
    assert checked > 4 * w.T


def test_training_step_graph_replays_match_eager():
    w = BLOCKS["bf16_shared"]
    lay, dv, dout, _, _ = _block(w)
    opt = moe.ExpertMuon(lay)
    start = {k: v.clone() for k, v in lay.w.items() if v is not None}

    def step():
        lay.forward(dv["x"])
        lay.backward(dout)
        opt.step(0.02)

    def reset():
        for k, v in start.items():
            lay.w[k].copy_(v)
        for m in opt.momentum.values():
            m.zero_()

    def state():
        return [t.clone() for t in (lay.out, lay.dx, lay.dnorm_gamma, lay.dnorm_beta,
                                    lay.dw_gate_up, *lay.w.values(), *opt.momentum.values())
                if t is not None]

    for _ in range(2):  # two steps: the second moves with momentum
        step()
    torch.cuda.synchronize()
    ref = state()
    reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        reset()
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, state()):
            assert torch.equal(a, b), f"replay {i}"
        lay.forward(dv["x"] * 0.5)  # eager work between replays
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    """A step of a rank that got no tokens: zero gradients, weights decayed."""
    w = wl.Workload("none", T=0, D=64, E=4, k=2, I=64, dtype=dtype, I_shared=64)
    lay, dv, dout, _, _ = _block(w)
    assert lay.forward(dv["x"]).shape == (0, 64)
    lay.backward(dout)
    names = ("dw_router", "dw_gate_up", "dw_down", "dw_shared_gate_up", "dw_shared_down",
             "dnorm_gamma", "dnorm_beta")
    assert not any(getattr(lay, k).any() for k in names)
    old = lay.w["w_down"].float().clone()
    moe.ExpertMuon(lay, weight_decay=0.5).step(0.5)
    torch.cuda.synchronize()
    assert torch.equal(lay.w["w_down"], (old * 0.75).to(w.torch_dtype))


def test_norm_arguments():
    d = moe.make_desc(T=4, D=64, E=2, top_k=1, I=64)
    t = torch.zeros(2, 64, 64, device="cuda")
    with pytest.raises(ValueError):
        moe.LayerTrain(d, t, t, t, norm_gamma=torch.ones(64, device="cuda"))
