"""LayerForwardFP8, and training steps of LayerTrain with 8-bit checkpoints and
the balance loss: against the same step without them, against the oracles, and
captured into a graph."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
import workloads as wl
from oracle import fp8_ckpt_balance_oracle as fo
from oracle import moe_oracle as om
from parity import np32, npi, to_dev

pytestmark = pytest.mark.gpu

LAYERS = {
    "shared": wl.Workload("ckpt_shared", T=200, D=128, E=8, k=2, I=192, I_shared=64),
    "plain": wl.Workload("ckpt_plain", T=333, D=192, E=20, k=3, I=64),
    "one": wl.Workload("ckpt_one", T=1, D=64, E=4, k=2, I=64, I_shared=128),
    "f32": wl.Workload("balance_f32", T=97, D=64, E=6, k=2, I=128, dtype="f32", I_shared=64),
}
BF16 = ["one", "plain", "shared"]


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


def inputs(w, seed=5):
    inp = wl.make_inputs(w, seed=seed)
    for k in ("w_gate_up", "w_down", "shared_gate_up", "shared_down"):
        if inp[k] is not None:
            inp[k] = (inp[k].float() * 5).to(inp[k].dtype)
    dv = to_dev(inp)
    g = torch.Generator().manual_seed(seed)
    return dv, torch.randn(w.T, w.D, generator=g).to(w.torch_dtype).cuda()


def layer(w, dv, **kw):
    d = moe.make_desc(T=w.T, D=w.D, E=w.E, top_k=w.k, I=w.I, I_shared=w.I_shared, dtype=w.dtype)
    return moe.LayerTrain(d, dv["w_router"], dv["w_gate_up"], dv["w_down"],
                          shared_gate_up=dv["shared_gate_up"], shared_down=dv["shared_down"], **kw)


def grads(lay):
    names = ["dx", "dw_router", "dw_gate_up", "dw_down", "dw_shared_gate_up", "dw_shared_down",
             "dnorm_gamma", "dnorm_beta"]
    return {k: getattr(lay, k) for k in names if getattr(lay, k, None) is not None}


def rel(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


# ---- the FP8 layer ----
@pytest.mark.parametrize("name", BF16)
def test_fp8_layer(name):
    w = LAYERS[name]
    dv, _ = inputs(w)
    d = moe.make_desc(T=w.T, D=w.D, E=w.E, top_k=w.k, I=w.I, I_shared=w.I_shared)
    args = (d, dv["w_router"], dv["w_gate_up"], dv["w_down"])
    sh = dict(shared_gate_up=dv["shared_gate_up"], shared_down=dv["shared_down"])
    lay = moe.LayerForwardFP8(*args, want_logits=True, **sh)
    out = lay(dv["x"]).clone()
    # The layer of the values that the codes stand for: rows and H are
    # quantized on the way, 2^-4 at most and 2.6 % in the mean of each value.
    def values(pair):
        v = fo.fp8_weight_values(pair[0].cpu().numpy(), pair[1].cpu().numpy())
        return v.transpose(0, 2, 1)
    more = {}
    if w.I_shared:
        more = dict(shared_gate_up=values(lay.sh_gate_up)[0], shared_down=values(lay.sh_down)[0])
    ref = om.layer_forward(np32(dv["x"]), np32(dv["w_router"]), values(lay.gate_up),
                           values(lay.down), w.k, **more)
    assert np.array_equal(npi(lay.topk_idx), ref["topk_idx"])
    branch = np32(out) - np32(dv["x"])
    want = ref["out"] - np32(dv["x"])
    # three quantizations of 2.6 % that add up like noise, and the output's own
    # rounding against a residual of about the branch's size
    assert np.linalg.norm(branch - want) <= 0.08 * np.linalg.norm(want) + 2.0 ** -9 * np.linalg.norm(
        np32(out))
    # given as codes and scales: the same bits
    pair = dict(shared_gate_up=lay.sh_gate_up, shared_down=lay.sh_down) if w.I_shared else {}
    again = moe.LayerForwardFP8(d, dv["w_router"], lay.gate_up, lay.down, **pair)
    assert torch.equal(again(dv["x"]), out)
    wide = moe.LayerForwardFP8(*args, y_fp16=False, **sh)
    assert rel(wide(dv["x"]), out) < 2e-3
    # replayed
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lay(dv["x"])
    x0 = dv["x"].clone()
    for i in range(3):
        dv["x"].copy_(torch.randn_like(x0))
        graph.replay()
        torch.cuda.synchronize()
        got = lay.out.clone()
        assert torch.equal(again(dv["x"]), got)


def test_fp8_layer_without_tokens():
    w = wl.Workload("none", T=0, D=64, E=4, k=2, I=64, dtype="bf16", I_shared=64)
    dv, _ = inputs(w)
    d = moe.make_desc(T=0, D=64, E=4, top_k=2, I=64, I_shared=64)
    lay = moe.LayerForwardFP8(d, dv["w_router"], dv["w_gate_up"], dv["w_down"],
                              shared_gate_up=dv["shared_gate_up"], shared_down=dv["shared_down"])
    assert lay(dv["x"]).shape == (0, 64)
    assert not lay.counts.any()


def test_fp8_layer_refuses_fp32():
    w = LAYERS["f32"]
    d = moe.make_desc(T=w.T, D=w.D, E=w.E, top_k=w.k, I=w.I, dtype="f32")
    with pytest.raises(ValueError, match="bf16"):
        moe.LayerForwardFP8(d, None, None, None)


# ---- 8-bit checkpoints ----
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("name", BF16)
def test_ckpt_step_against_the_plain_one(name, norm):
    w = LAYERS[name]
    dv, dout = inputs(w)
    plain, kept = layer(w, dv, norm=norm), layer(w, dv, norm=norm, ckpt=True)
    a, b = plain.forward(dv["x"]), kept.forward(dv["x"])
    assert torch.equal(a, b) and kept.gu is None
    x_perm, y_perm = kept.x_perm.clone(), kept.y_perm.clone()
    # nothing but the 8-bit copies is left
    for t in (kept.x_perm, kept.y_perm, kept.x_back, kept.dx_perm, kept.dy_perm):
        t.fill_(float("nan"))
    if norm:
        kept.h.fill_(float("nan"))
    plain.backward(dout)
    kept.backward(dout)
    torch.cuda.synchronize()
    # What came back is the rows to 1/254 of each block's largest value.
    for got, want in ((kept.x_perm, x_perm), (kept.y_perm, y_perm)):
        blocks = want.float().reshape(-1, 32)
        top = blocks.abs().amax(1, keepdim=True)
        assert ((got.float().reshape(-1, 32) - blocks).abs()
                <= top * (0.5 / 127 * 1.01 + 2.0 ** -8)).all()
    # Gradients move by the checkpoints' own error: 0.5 to 1 % of each factor
    # in the mean (uniform within half a step of 1/127 of a block's largest
    # value, some 2.5 standard deviations), two to three factors.
    for k, want in grads(plain).items():
        got = grads(kept)[k]
        assert torch.isfinite(got).all(), k
        assert rel(got, want) < 0.03, (k, rel(got, want))


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("ckpt", [False, True])
def test_no_tokens(ckpt, norm):
    """A step of a rank that got no tokens: zero gradients, zero loss."""
    w = wl.Workload("none", T=0, D=64, E=4, k=2, I=64, dtype="bf16", I_shared=64)
    dv, dout = inputs(w)
    lay = layer(w, dv, ckpt=ckpt, norm=norm, balance=0.1)
    lay.balance_loss.fill_(7.0)
    for g in grads(lay).values():
        g.fill_(7.0)
    assert lay.forward(dv["x"]).shape == (0, 64)
    lay.backward(dout)
    assert lay.balance_loss.item() == 0 and lay.balance_tokens.item() == 0
    assert not lay.balance_counts.any() and not lay.balance_prob_sum.any()
    assert not any(g.any() for g in grads(lay).values())


def test_layers_that_share_scratch():
    """Two layers one after another through one scratch: the gradients of each
    are those it has with scratch of its own."""
    w = LAYERS["shared"]
    alone, together, pool = [], [], {}
    ins = [inputs(w, seed=s) for s in (5, 6)]
    for dv, dout in ins:
        lay = layer(w, dv, ckpt=True, norm=True, balance=0.01)
        lay.forward(dv["x"])
        lay.backward(dout)
        alone.append({k: v.clone() for k, v in grads(lay).items()})
    lays = [layer(w, dv, ckpt=True, norm=True, balance=0.01, scratch=pool) for dv, _ in ins]
    assert lays[0].x_perm.data_ptr() == lays[1].x_perm.data_ptr()
    for lay, (dv, _) in zip(lays, ins):
        lay.forward(dv["x"])
    for i in (1, 0):
        lays[i].backward(ins[i][1])
        together.insert(0, {k: v.clone() for k, v in grads(lays[i]).items()})
    for a, b in zip(alone, together):
        for k in a:
            assert torch.equal(a[k], b[k]), k
    with pytest.raises(ValueError, match="other sizes"):
        layer(LAYERS["plain"], inputs(LAYERS["plain"])[0], ckpt=True, scratch=pool)


def test_ckpt_refusals():
    w = LAYERS["f32"]
    dv, _ = inputs(w)
    with pytest.raises(ValueError, match="bf16"):
        layer(w, dv, ckpt=True)
    w = LAYERS["plain"]
    dv, dout = inputs(w)
    with pytest.raises(ValueError, match="save_gu"):
        layer(w, dv, ckpt=True, save_gu=True)
    with pytest.raises(ValueError, match="scratch"):
        layer(w, dv, scratch={})
    lay = layer(w, dv)
    with pytest.raises(ValueError, match="balance"):
        lay.forward(dv["x"], mask=torch.ones(w.T, dtype=torch.bool, device="cuda"))
    lay.forward(dv["x"])
    with pytest.raises(ValueError, match="balance"):
        lay.backward(dout, dloss=torch.ones(1, device="cuda"))


# ---- the balance loss ----
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("name", sorted(LAYERS))
def test_balance_step(name, norm):
    w = LAYERS[name]
    dv, dout = inputs(w)
    coef = 0.5
    mask = (torch.arange(w.T) % 7 != 3).cuda()
    plain, zero = layer(w, dv, norm=norm), layer(w, dv, norm=norm, balance=0.0)
    lay = layer(w, dv, norm=norm, balance=coef)
    outs = [plain.forward(dv["x"]), zero.forward(dv["x"], mask=mask),
            lay.forward(dv["x"], mask=mask)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    z, topk, m = np32(lay.logits).astype(np.float64), npi(lay.topk_idx), mask.cpu().numpy()
    counts, n, prob, loss = fo.balance_loss(z, topk, coef, m)
    assert np.array_equal(npi(lay.balance_counts), counts) and int(lay.balance_tokens) == n
    assert abs(float(lay.balance_loss) - loss) <= 1e-5 * loss
    dloss = torch.tensor([3.0], device="cuda")
    plain.backward(dout)
    zero.backward(dout, dloss=dloss)
    lay.backward(dout, dloss=dloss)
    torch.cuda.synchronize()
    ga, gz, gb = grads(plain), grads(zero), grads(lay)
    tol = 1e-5 if w.dtype == "f32" else 2e-2
    for k in ga:
        if k.startswith("dw_") and k != "dw_router":
            assert torch.equal(ga[k], gz[k]) and torch.equal(ga[k], gb[k]), k
    # coefficient 0: the dense way gives the sparse way's gradient
    assert rel(gz["dw_router"], ga["dw_router"]) < 1e-5
    assert rel(gz["dx"], ga["dx"]) < tol
    # the balance term: dlogits from the oracle, through x and W_r
    d = fo.balance_backward(z, coef, w.k, counts, n, 3.0, m)
    x = np32(lay.h if norm else dv["x"]).astype(np.float64)
    got = (gb["dw_router"] - gz["dw_router"]).double().cpu().numpy()
    want = d.T @ x
    # the difference of two fp32 sums, each rounded at its own size
    own = np.abs(np32(gz["dw_router"])).max() + np.abs(want).max()
    assert np.abs(got - want).max() <= 1e-5 * own * np.sqrt(w.T)
    if not norm and w.dtype == "f32":
        got = (gb["dx"] - gz["dx"]).double().cpu().numpy()
        want = d @ np32(dv["w_router"]).astype(np.float64)
        assert np.abs(got - want).max() <= 1e-5 * np.abs(np32(gb["dx"])).max()


def test_router_gradient_against_differences():
    """dW_r of sum(out dout) + balance loss, fp32 layer, against central
    differences of the float64 oracles (the choice of experts held)."""
    w = LAYERS["f32"]
    dv, dout = inputs(w, seed=8)
    coef = 2.0
    lay = layer(w, dv, balance=coef)
    lay.forward(dv["x"])
    lay.backward(dout)
    torch.cuda.synchronize()
    x, wr = np32(dv["x"]).astype(np.float64), np32(dv["w_router"]).astype(np.float64)
    idx, do = npi(lay.topk_idx), np32(dout).astype(np.float64)
    rest = [np32(dv[k]).astype(np.float64) for k in ("w_gate_up", "w_down")]
    y = np.stack([fo.silu(x @ rest[0][e][:, :w.I]) * (x @ rest[0][e][:, w.I:]) @ rest[1][e]
                  for e in range(w.E)])

    def loss(wr):
        z = x @ wr.T
        zk = np.take_along_axis(z, idx, 1)
        p = np.exp(zk - zk.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out = sum(p[:, j:j + 1] * y[idx[:, j], np.arange(w.T)] for j in range(w.k))
        return (out * do).sum() + fo.balance_loss(z, idx, coef)[3]

    got = lay.dw_router.double().cpu().numpy()
    h = 1e-5
    g = np.random.default_rng(0)
    for _ in range(25):
        e, c = g.integers(w.E), g.integers(w.D)
        dw = np.zeros_like(wr)
        dw[e, c] = h
        num = (loss(wr + dw) - loss(wr - dw)) / (2 * h)
        assert abs(num - got[e, c]) <= 2e-5 * np.abs(got).max() + 1e-6


def test_whole_step_replayed():
    """Norm, checkpoints and balance loss in one captured step, replayed on new
    inputs with eager steps between."""
    w = LAYERS["shared"]
    dv, dout = inputs(w)
    lay = layer(w, dv, norm=True, ckpt=True, balance=0.01)

    def step():
        lay.forward(dv["x"])
        lay.backward(dout)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        dv["x"].copy_(torch.randn(w.T, w.D, device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in grads(lay).items()}
        got["loss"] = lay.balance_loss.clone()
        step()
        torch.cuda.synchronize()
        for k, v in grads(lay).items():
            assert torch.equal(got[k], v), k
        assert torch.equal(got["loss"], lay.balance_loss)


# ---- two streams at once ----
def test_calls_on_two_streams_at_once():
    """Layers with buffers of their own, stepped on two streams side by side:
    the bits of steps one after another."""
    w = LAYERS["shared"]
    runs = []
    for seed in (5, 6):
        dv, dout = inputs(w, seed)
        d = moe.make_desc(T=w.T, D=w.D, E=w.E, top_k=w.k, I=w.I, I_shared=w.I_shared)
        fp8 = moe.LayerForwardFP8(d, dv["w_router"], dv["w_gate_up"], dv["w_down"],
                                  shared_gate_up=dv["shared_gate_up"],
                                  shared_down=dv["shared_down"])
        lay = layer(w, dv, ckpt=True, balance=0.1, norm=True)

        def step(stream=None, dv=dv, dout=dout, fp8=fp8, lay=lay):
            fp8(dv["x"], stream)
            lay.forward(dv["x"], stream)
            lay.backward(dout, stream)

        def results(fp8=fp8, lay=lay):
            return [t.clone() for t in (fp8.out, lay.out, lay.balance_loss, *grads(lay).values())]

        runs.append((step, results))
    want = []
    for step, results in runs:
        step()
        want.append(results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for (step, _), s in zip(runs, streams):
            step(s)
    torch.cuda.synchronize()
    for (_, results), ref in zip(runs, want):
        assert all(torch.equal(a, b) for a, b in zip(results(), ref))
