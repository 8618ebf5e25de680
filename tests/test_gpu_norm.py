"""Layer norm forward and backward on the GPU against the float64 oracle.

Tolerances, with u = 2^-24 (a rounding in fp32). A row's sum goes through at
most 16 adds in a thread, 6 across a wave and 16 across waves (wide rows: up to
256 more in a thread), so a mean over it is off by at most S u mean|.|, S = 40
(300). h = (x - mean) rstd then has an error below
  S u (|x| + mean|x|) rstd + |h| (S + 4) u,
y adds two roundings and its own type's, dx the errors of its two row means
(each term times rstd), and a column sum over R rows at most R + 40 roundings of
its terms (in practice far fewer; the sum is taken in parts).
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from oracle import norm_update_oracle as ou

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


def _roundings(D):
    return 40 if D <= 16384 else 300


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _inputs(rows, D, dt, seed=0, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (r(rows, D) * torch.exp(0.5 * r(rows, 1)) + offset * r(D)).to(dt)
    return dict(x=x.cuda(), gamma=(1 + 0.2 * r(D)).cuda(), beta=(0.3 * r(D)).cuda(),
                dy=r(rows, D).to(dt).cuda(), dres=r(rows, D).to(dt).cuda())


def _h_error(x, mean, rstd, D):
    s = _roundings(D)
    h = (x - mean[:, None]) * rstd[:, None]
    ax = np.abs(x)
    return h, (s * U * (ax + ax.mean(1, keepdims=True)) * rstd[:, None]
               + np.abs(h) * (s + 4) * U)


def _forward(i, gamma, beta, eps=1e-5):
    x = i["x"]
    y = torch.full_like(x, 7.0)
    mean, rstd = torch.empty(2, x.shape[0], device="cuda")
    moe.moe_layer_norm(x, gamma, beta, eps, y, mean, rstd)
    torch.cuda.synchronize()
    return y, mean, rstd


SIZES = [(1, 1), (1, 64), (3, 7), (5, 128), (257, 64), (2, 1024), (9, 1000), (130, 1031),
         (3, 2048), (65, 2050), (2, 4096), (300, 4095), (4, 7168), (3, 8200), (2, 16384),
         (2, 16385), (3, 40000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", SIZES)
def test_forward(rows, D, dtype):
    print(f"[norm] forward rows={rows} D={D} {dtype}", flush=True)
    dt = DT[dtype]
    i = _inputs(rows, D, dt)
    x, gm, bt = _np(i["x"]), _np(i["gamma"]), _np(i["beta"])
    for gamma, beta in ((i["gamma"], i["beta"]), (None, None), (i["gamma"], None)):
        y, mean, rstd = _forward(i, gamma, beta)
        ry, rm, rr = ou.layer_norm(x, _np(gamma), _np(beta))
        assert np.all(np.abs(_np(mean) - rm) <= _roundings(D) * U * np.abs(x).mean(1))
        h, eh = _h_error(x, rm, rr, D)
        # rstd: half the relative error of the variance, and its own roundings
        ev = 2 * (np.abs(h) * eh).mean(1) + (_roundings(D) + 8) * U
        assert np.all(np.abs(_np(rstd) - rr) <= rr * ev)
        tol = ((eh + np.abs(h) * ev[:, None]) * np.abs(gm if gamma is not None else 1.0)
               + 3 * U * (np.abs(ry) + np.abs(bt if beta is not None else 0.0))
               + HALF[dt] * np.abs(ry))
        assert np.all(np.abs(_np(y) - ry) <= tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", SIZES + [(5000, 128), (2600, 2048)])
def test_backward(rows, D, dtype):
    print(f"[norm] backward rows={rows} D={D} {dtype}", flush=True)
    dt = DT[dtype]
    i = _inputs(rows, D, dt, seed=1)
    x, dy, gm, res = _np(i["x"]), _np(i["dy"]), _np(i["gamma"]), _np(i["dres"])
    _, mean, rstd = ou.layer_norm(x)
    # The statistics as the forward leaves them: fp32 values.
    mt, rt = (torch.from_numpy(v).float().cuda() for v in (mean, rstd))
    mean, rstd = _np(mt), _np(rt)
    ws = moe.workspace(moe.moe_layer_norm_backward_workspace_size(rows, D))
    s = _roundings(D)
    for gamma, dres, params in ((i["gamma"], i["dres"], True), (None, None, True),
                                (i["gamma"], None, False)):
        dx = torch.full_like(i["x"], 7.0)
        dgamma, dbeta = torch.full((2, D), 7.0, device="cuda") if params else (None, None)
        moe.moe_layer_norm_backward(i["x"], i["dy"], gamma, mt, rt, dres, dx, dgamma, dbeta,
                                    ws if params else None)
        torch.cuda.synchronize()
        rdx, rdg, rdb = ou.layer_norm_backward(x, dy, _np(gamma), mean, rstd, _np(dres))
        h = (x - mean[:, None]) * rstd[:, None]
        eh = 2 * U * (np.abs(x) + np.abs(mean)[:, None]) * rstd[:, None] + np.abs(h) * U
        g = np.abs(dy * (gm if gamma is not None else 1.0))
        c1 = np.abs((g * np.abs(h))).mean(1, keepdims=True)
        e1 = ((g * eh).mean(1, keepdims=True) + (s + 3) * U * c1)
        tol = rstd[:, None] * (6 * U * (g + g.mean(1, keepdims=True) + np.abs(h) * c1)
                               + s * U * g.mean(1, keepdims=True) + np.abs(h) * e1 + eh * c1)
        tol += (HALF[dt] + 2 * U) * np.abs(rdx)
        if dres is not None:
            tol += 2 * U * np.abs(res)
        assert np.all(np.abs(_np(dx) - rdx) <= tol)
        if params:
            a = np.abs(dy)
            assert np.all(np.abs(_np(dgamma) - rdg)
                          <= (a * eh).sum(0) + (rows + 40) * U * (a * np.abs(h)).sum(0))
            assert np.all(np.abs(_np(dbeta) - rdb) <= (rows + 40) * U * a.sum(0))


def test_gradient_against_differences():
    """dx, dgamma and dbeta of the kernels against differences of the oracle's
    forward (float64): the kernels' fp32 error is far below the 1e-5 allowed."""
    i = _inputs(3, 40, torch.float32, seed=3)
    x, gm, bt, dy = (_np(i[k]) for k in ("x", "gamma", "beta", "dy"))
    _, mean, rstd = _forward(i, i["gamma"], i["beta"])
    dx = torch.empty_like(i["x"])
    dgamma, dbeta = torch.empty(2, 40, device="cuda")
    ws = moe.workspace(moe.moe_layer_norm_backward_workspace_size(3, 40))
    moe.moe_layer_norm_backward(i["x"], i["dy"], i["gamma"], mean, rstd, None, dx, dgamma, dbeta,
                                ws)
    loss = lambda x, g, b: (ou.layer_norm(x, g, b)[0] * dy).sum()  # noqa: E731
    step = 1e-5
    for at in ((0, 0), (1, 17), (2, 39)):
        e = np.zeros_like(x)
        e[at] = step
        d = (loss(x + e, gm, bt) - loss(x - e, gm, bt)) / (2 * step)
        assert abs(d - float(dx[at])) <= 1e-5 * (1 + abs(d))
    for j in (0, 21, 39):
        e = np.zeros(40)
        e[j] = step
        d = (loss(x, gm + e, bt) - loss(x, gm - e, bt)) / (2 * step)
        assert abs(d - float(dgamma[j])) <= 1e-5 * (1 + abs(d))
        d = (loss(x, gm, bt + e) - loss(x, gm, bt - e)) / (2 * step)
        assert abs(d - float(dbeta[j])) <= 1e-5 * (1 + abs(d))


def test_rows_with_nan_inf_and_constant_rows():
    i = _inputs(6, 300, torch.float32, seed=4)
    x = i["x"]
    clean, _, _ = _forward(i, i["gamma"], i["beta"])
    x[1, 5] = float("nan")
    x[3, 299] = float("inf")
    x[4] = 2.5  # variance 0
    y, mean, rstd = _forward(i, i["gamma"], i["beta"])
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    assert torch.equal(y[4], i["beta"]) and abs(float(rstd[4]) - 1e5 ** 0.5) < 1e-3
    for r in (0, 2, 5):
        assert torch.equal(y[r], clean[r])


def test_no_rows():
    D = 96
    x = torch.empty(0, D, device="cuda")
    moe.moe_layer_norm(x, None, None, 1e-5, torch.empty_like(x))
    dgamma, dbeta = torch.full((2, D), 3.0, device="cuda")
    st = torch.empty(0, device="cuda")
    moe.moe_layer_norm_backward(x, x.clone(), None, st, st.clone(), None, x.clone(), dgamma, dbeta,
                                moe.workspace(0))
    assert not dgamma.any() and not dbeta.any()


@pytest.mark.parametrize("D", [64, 1031])
def test_neighbours_stay_and_offsets_work(D):
    """Rows inside a larger buffer, starting at an odd element: the values
    around the written rows stay."""
    rows, lead = 5, 3
    for dt in (torch.float32, torch.bfloat16):
        i = _inputs(rows, D, dt, seed=5)
        buf = lambda: torch.full((lead + rows * D + 9,), 11.0, dtype=dt, device="cuda")  # noqa
        bx, by, bd, bo = buf(), buf(), buf(), buf()
        view = lambda b: b[lead:lead + rows * D].view(rows, D)  # noqa: E731
        view(bx).copy_(i["x"])
        view(bd).copy_(i["dy"])
        mean, rstd = torch.empty(2, rows, device="cuda")
        moe.moe_layer_norm(view(bx), i["gamma"], i["beta"], 1e-5, view(by), mean, rstd)
        ref, m2, r2 = _forward(i, i["gamma"], i["beta"])
        assert torch.equal(view(by), ref)
        ws = moe.workspace(moe.moe_layer_norm_backward_workspace_size(rows, D))
        dgb = torch.full((2, D + 2), 11.0, device="cuda")
        moe.moe_layer_norm_backward(view(bx), view(bd), i["gamma"], mean, rstd, None, view(bo),
                                    dgb[0, 1:D + 1], dgb[1, 1:D + 1], ws)
        dx = torch.empty_like(i["x"])
        dg, db = torch.empty(2, D, device="cuda")
        moe.moe_layer_norm_backward(i["x"], i["dy"], i["gamma"], m2, r2, None, dx, dg, db, ws)
        assert torch.equal(view(bo), dx)
        assert torch.equal(dgb[0, 1:D + 1], dg) and torch.equal(dgb[1, 1:D + 1], db)
        for b in (by, bo):
            assert (b[:lead] == 11).all() and (b[lead + rows * D:] == 11).all()
        assert (dgb[:, 0] == 11).all() and (dgb[:, -1] == 11).all()


def test_same_bits_on_another_stream_and_in_a_graph():
    rows, D = 700, 2050
    i = _inputs(rows, D, torch.bfloat16, seed=6)
    ws = moe.workspace(moe.moe_layer_norm_backward_workspace_size(rows, D))
    y, dx = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    stats = torch.empty(2, rows, device="cuda")
    par = torch.empty(2, D, device="cuda")

    def step():
        moe.moe_layer_norm(i["x"], i["gamma"], i["beta"], 1e-5, y, stats[0], stats[1])
        moe.moe_layer_norm_backward(i["x"], i["dy"], i["gamma"], stats[0], stats[1], i["dres"],
                                    dx, par[0], par[1], ws)

    step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (y, dx, stats, par)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, (y, dx, stats, par)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in (y, dx, stats, par):
            t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, (y, dx, stats, par)))
        step()  # eager work between replays
        torch.cuda.synchronize()
