"""Cases that measure the layer norm, the orthogonalisation and the Muon update.

A case's ``op`` names the operator:

``norm``       moe_layer_norm: y, mean, rstd of x [rows, D].
``norm_bwd``   moe_layer_norm_backward: dx (with the residual's gradient added
               when ``res``), dgamma, dbeta.
``orth``       moe_orthogonalize: the Newton-Schulz iteration on n matrices.
``muon``       moe_muon_update: momentum, orthogonalisation and the update of
               n weight matrices, in place. With ``half`` the matrices are the
               gate columns of gate | up tensors [n, rows, 2 cols].

``run`` computes the plain form with elementary torch operations in 32 bits
(norms of whole matrices in 64), or, when ``own`` is true, calls the package.
"""
import math

import torch

own = False

EPS_NORM = 1e-5    # layer norm
EPS_ORTH = 1e-7    # added to the Frobenius norm
STEPS = 5
COEFS = (3.4445, -4.7750, 2.0315)
MUON = dict(lr=0.02, mu=0.95, weight_decay=0.01)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # One new token of the rank-share layer's width in front of the router: a launch's latency.
        dict(name="norm_token", op="norm", rows=1, D=7168, dtype="bf16"),
        # Every token of the Mixtral-style layer's forward.
        dict(name="norm_mixtral_style", op="norm", rows=8192, D=4096, dtype="bf16"),
        # A ragged batch of a width that no vector load divides, fp32 layer.
        dict(name="norm_odd", op="norm", rows=777, D=1031, dtype="f32"),
        # The tiny fp32 layer's training step.
        dict(name="norm_bwd_tiny", op="norm_bwd", rows=256, D=128, dtype="f32", res=False),
        # The fine-grained layer's training step, the residual branch joined in: many rows to reduce.
        dict(name="norm_bwd_skewed", op="norm_bwd", rows=16384, D=2048, dtype="bf16", res=True),
        # The rank-share layer's own tokens in fp32: the widest rows.
        dict(name="norm_bwd_wide", op="norm_bwd", rows=4096, D=7168, dtype="f32", res=True),
        # gate_up gradients of the tiny fp32 layer: launches count.
        dict(name="orth_tiny", op="orth", n=8, rows=128, cols=512, dtype="f32"),
        # Odd sizes, taller than wide.
        dict(name="orth_odd", op="orth", n=3, rows=1001, cols=333, dtype="bf16"),
        # down_proj of one Mixtral-style expert: the largest products.
        dict(name="orth_mixtral_style", op="orth", n=1, rows=14336, cols=4096, dtype="bf16"),
        # down_proj of the tiny fp32 layer's eight experts.
        dict(name="muon_tiny", op="muon", n=8, rows=256, cols=128, dtype="f32", half=False),
        # Gate columns of the worked example's sixteen experts.
        dict(name="muon_worked_example", op="muon", n=16, rows=1024, cols=2048, dtype="bf16",
             half=True),
        # down_proj of the fine-grained layer: 128 small experts at once.
        dict(name="muon_skewed", op="muon", n=128, rows=768, cols=2048, dtype="bf16", half=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """Token batches from one row to the longest listed, widths from 32 up;
    one to 64 matrices with sides from 24 to 4096, within the listed cost."""
    op = rng.choice(["norm", "norm_bwd", "orth", "muon"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    if op in ("norm", "norm_bwd"):
        D = _log_int(rng, 32, 8192)
        if rng.random() < 0.5:
            D = max(64, D // 64 * 64)
        rows = _log_int(rng, 1, min(16384, 4096 * 7168 // D))
        case = dict(op=op, rows=rows, D=D, dtype=dtype)
        if op == "norm_bwd":
            case["res"] = rng.random() < 0.5
        return case
    rows, cols = _log_int(rng, 24, 4096), _log_int(rng, 24, 4096)
    if rng.random() < 0.5:
        rows, cols = max(64, rows // 64 * 64), max(64, cols // 64 * 64)
    most = 128 * 768 * 2048
    n = _log_int(rng, 1, max(1, min(64, most // (rows * cols))))
    case = dict(op=op, n=n, rows=rows, cols=cols, dtype=dtype)
    if op == "muon":
        case["half"] = rng.random() < 0.5
    return case


def _gradient(n, rows, cols, g, dev):
    """fp32 gradients of n experts' matrices: X^T dY over the expert's tokens
    (more tokens than the short side), rows of X of uneven size."""
    tokens = min(rows, cols) + min(rows, cols) // 2 + 8
    x = torch.randn(n, tokens, rows, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(n, tokens, 1, generator=g, device=dev))
    dy = torch.randn(n, tokens, cols, generator=g, device=dev)
    return torch.matmul(x.transpose(1, 2).contiguous(), dy) * (1e-3 / math.sqrt(tokens))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DT[case["dtype"]]
    st = {"case": case}
    if case["op"] in ("norm", "norm_bwd"):
        rows, D = case["rows"], case["D"]
        # Hidden states: rows of uneven scale, some features far from zero.
        x = torch.randn(rows, D, generator=g, device=dev)
        x *= torch.exp(0.3 * torch.randn(rows, 1, generator=g, device=dev))
        x += torch.randn(D, generator=g, device=dev) * 0.5
        st["x"] = x.to(dt)
        st["gamma"] = 1 + 0.1 * torch.randn(D, generator=g, device=dev)
        st["beta"] = 0.1 * torch.randn(D, generator=g, device=dev)
        if case["op"] == "norm":
            if own:
                st["y"] = torch.empty_like(st["x"])
                st["mean"] = torch.empty(rows, device=dev)
                st["rstd"] = torch.empty(rows, device=dev)
            return st
        st["dy"] = torch.randn(rows, D, generator=g, device=dev).to(dt)
        st["dres"] = (torch.randn(rows, D, generator=g, device=dev).to(dt) if case["res"]
                      else None)
        # What the forward pass has left.
        xd = st["x"].double()
        mean = xd.mean(1)
        st["mean"] = mean.float()
        st["rstd"] = ((xd - mean[:, None]).square().mean(1) + EPS_NORM).rsqrt().float()
        if own:
            import mixture_experts_layer_fp32_amd as moe
            st["dx"] = torch.empty_like(st["x"])
            st["dgamma"], st["dbeta"] = torch.empty(2, D, device=dev)
            st["ws"] = moe.workspace(moe.moe_layer_norm_backward_workspace_size(rows, D), dev)
        return st
    n, rows, cols = case["n"], case["rows"], case["cols"]
    if case["op"] == "orth":
        st["g"] = _gradient(n, rows, cols, g, dev)
        if own:
            st["out"] = torch.empty(n, rows, cols, dtype=dt, device=dev)
    else:
        wide = 2 * cols if case["half"] else cols
        st["full_g"] = torch.cat([_gradient(n, rows, cols, g, dev) for _ in range(wide // cols)], 2)
        st["full_m"] = (torch.cat([_gradient(n, rows, cols, g, dev)
                                   for _ in range(wide // cols)], 2) * 3)
        st["full_w"] = (torch.randn(n, rows, wide, generator=g, device=dev) * 0.02).to(dt)
        for k in ("g", "m", "w"):
            st[k] = st["full_" + k][:, :, :cols]
        st["scale"] = 0.2 * math.sqrt(max(rows, cols))
    if own:
        import mixture_experts_layer_fp32_amd as moe
        st["ws"] = moe.workspace(moe.moe_orthogonalize_workspace_size(n, rows, cols, STEPS), dev)
    return st


def _norm_plain(st):
    x = st["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = (xc.square().mean(1) + EPS_NORM).rsqrt()
    y = xc * rstd[:, None] * st["gamma"] + st["beta"]
    return {"y": y.to(st["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_bwd_plain(st):
    h = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
    dy = st["dy"].float()
    gg = dy * st["gamma"]
    dx = (gg - gg.mean(1, keepdim=True) - h * (gg * h).mean(1, keepdim=True)) * st["rstd"][:, None]
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(st["x"].dtype), "dgamma": (dy * h).sum(0), "dbeta": dy.sum(0)}


def _orth_plain(u):
    norm = u.double().square().sum((1, 2), keepdim=True).sqrt() + EPS_ORTH
    x = (u / norm).float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    a, b, c = COEFS
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return x.transpose(1, 2).contiguous() if tall else x


def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        import mixture_experts_layer_fp32_amd as moe
        if op == "norm":
            moe.moe_layer_norm(state["x"], state["gamma"], state["beta"], EPS_NORM, state["y"],
                               state["mean"], state["rstd"])
            return {k: state[k] for k in ("y", "mean", "rstd")}
        if op == "norm_bwd":
            moe.moe_layer_norm_backward(state["x"], state["dy"], state["gamma"], state["mean"],
                                        state["rstd"], state["dres"], state["dx"],
                                        state["dgamma"], state["dbeta"], state["ws"])
            return {k: state[k] for k in ("dx", "dgamma", "dbeta")}
        if op == "orth":
            moe.moe_orthogonalize(state["g"], state["out"], state["ws"], steps=STEPS, eps=EPS_ORTH)
            return {"out": state["out"]}
        moe.moe_muon_update(state["g"], state["m"], state["w"], state["ws"], scale=state["scale"],
                            nesterov=True, steps=STEPS, eps=EPS_ORTH, **MUON)
        return {"momentum": state["full_m"], "w": state["full_w"]}
    if op == "norm":
        return _norm_plain(state)
    if op == "norm_bwd":
        return _norm_bwd_plain(state)
    if op == "orth":
        return {"out": _orth_plain(state["g"]).to(DT[case["dtype"]])}
    mu, lr = MUON["mu"], MUON["lr"]
    state["m"].mul_(mu).add_(state["g"])
    o = _orth_plain(state["g"] + mu * state["m"])
    state["w"].copy_(state["w"].float() * (1 - lr * MUON["weight_decay"])
                     - (lr * state["scale"]) * o)
    return {"momentum": state["full_m"], "w": state["full_w"]}


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("norm", "norm_bwd"):
        v = case["rows"] * case["D"]
        if case["op"] == "norm":
            return {"bytes": 2 * v * es + 8 * case["D"] + 8 * case["rows"], "flops": 8 * v}
        passes = 4 if case["res"] else 3
        return {"bytes": passes * v * es + 12 * case["D"] + 8 * case["rows"], "flops": 14 * v}
    n, rows, cols = case["n"], case["rows"], case["cols"]
    v, m, k = n * rows * cols, min(rows, cols), max(rows, cols)
    # X X^T and what follows it are symmetric: half a product each. Step by
    # step: X X^T, A^2 and P X; or one X X^T, the steps on the short side
    # alone (A^2, then A P, P A P, A^2, P Q a step) and one product with X.
    direct = STEPS * (3 * k * m * m + m ** 3)
    short = 3 * k * m * m + (1 + 4 * (STEPS - 1)) * m ** 3
    flops = n * min(direct, short)
    if case["op"] == "orth":
        return {"bytes": v * (4 + es), "flops": flops}
    return {"bytes": v * (4 + 8 + 2 * es), "flops": flops}


def exact(case, seed):
    st = prepare(case, seed)
    x64 = {k: t.double() for k, t in st.items() if torch.is_tensor(t) and t.is_floating_point()}
    if case["op"] == "norm":
        var, mean = torch.var_mean(x64["x"], dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS_NORM)
        y = torch.addcmul(x64["beta"], (x64["x"] - mean.unsqueeze(1)) * rstd.unsqueeze(1),
                          x64["gamma"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if case["op"] == "norm_bwd":
        r = x64["rstd"].unsqueeze(1)
        h = (x64["x"] - x64["mean"].unsqueeze(1)) * r
        w, D = x64["dy"] * x64["gamma"], case["D"]
        s1, s2 = w.sum(1, keepdim=True), (w * h).sum(1, keepdim=True)
        dx = r / D * (D * w - s1 - h * s2)
        if case["res"]:
            dx = dx + x64["dres"]
        return {"dx": dx, "dgamma": torch.einsum("td,td->d", x64["dy"], h),
                "dbeta": x64["dy"].sum(0)}

    def polar(u):
        # The polynomial on the right side or the left, whichever is short.
        p = u / (torch.linalg.matrix_norm(u) + EPS_ORTH)[:, None, None]
        eye = torch.eye(min(p.shape[1:]), dtype=p.dtype, device=p.device)
        for _ in range(STEPS):
            right = p.shape[1] > p.shape[2]
            s = p.mT @ p if right else p @ p.mT
            q = COEFS[0] * eye + s @ (COEFS[1] * eye + COEFS[2] * s)
            p = p @ q if right else q @ p
        return p

    if case["op"] == "orth":
        return {"out": polar(x64["g"])}
    mom = MUON["mu"] * x64["m"] + x64["g"]
    o = polar(x64["g"] + MUON["mu"] * mom)
    full_m, full_w = x64["full_m"], x64["full_w"]
    full_m[:, :, :case["cols"]] = mom
    full_w[:, :, :case["cols"]] = ((1 - MUON["lr"] * MUON["weight_decay"]) * x64["w"]
                                   - MUON["lr"] * st["scale"] * o)
    return {"momentum": full_m, "w": full_w}
