"""The calls around a layer, and the layer with an epilogue, on tensors whose offsets pass 2^31 values: rows at both ends and around the
2^31st value against 64 bits, sums over all rows in pieces."""
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests import layer_reference as lr
from tests import test_gpu_act as ta
from tests import test_gpu_norm as tn

pytestmark = pytest.mark.gpu
u = 2.0 ** -24


def random(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def rows_to_look_at(n, w):
    edge = 2 ** 31 // w
    return torch.tensor([0, 1, n // 2, edge - 1, edge, edge + 1, n - 2, n - 1], device="cuda")


def test_norm():
    n, w = 525_000, 4104
    assert n * w > 2 ** 31
    look = rows_to_look_at(n, w)
    c = tn.Case(3, "bf16", len(look), w)
    X, dY, beyond = random(1, n, w), random(2, n, w), random(3, n, w)
    c.X, c.dY, c.beyond = X[look], dY[look], beyond[look]
    Y, mean, rstd = torch.empty_like(X), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    sg.sgmv_layer_norm_apply(X, c.gamma, c.beta, Y, c.eps, mean=mean, rstd=rstd)
    for got, (ref, bound), what in zip((Y[look], mean[look], rstd[look]), c.ref_forward(), ("Y", "mean", "rstd")):
        tn.check(got, ref, bound, what)
    dg, db = torch.empty_like(c.gamma), torch.empty_like(c.beta)
    sg.sgmv_layer_norm_backward(X, c.gamma, mean, rstd, dY, sg.new_layer_norm_workspace(n, w), dX=Y, beyond=beyond, dgamma=dg, dbeta=db)
    tn.check(Y[look], *c.ref_backward(mean[look], rstd[look])[0], "dX")
    sums = torch.zeros(4, w, dtype=torch.float64, device="cuda")
    for i in range(0, n, 20_000):
        xh = (X[i:i + 20_000].double() - mean[i:i + 20_000, None].double()) * rstd[i:i + 20_000, None].double()
        dy = dY[i:i + 20_000].double()
        sums += torch.stack([(dy * xh).sum(0), (dy * xh).abs().sum(0), dy.sum(0), dy.abs().sum(0)])
    deep = n // 512 + 80
    tn.check(dg, sums[0], deep * u * sums[1], "dgamma")
    tn.check(db, sums[2], deep * u * sums[3], "dbeta")


def test_rows_out_and_back():
    n, k, w = 265_000, 2, 4104
    m = n * k
    assert m * w > 2 ** 31
    ids = torch.randint(-1, 7, (n, k), device="cuda", dtype=torch.int32)
    slots, weights = torch.empty(m, dtype=torch.int32, device="cuda"), torch.rand(n, k, device="cuda")
    sg.sgmv_route_rows(ids, 7, None, slots, None, None, sg.new_route_workspace(n, k, 7))
    at = slots.long().reshape(n, k)
    X, Xs = random(4, n, w), torch.empty(m, w, dtype=torch.bfloat16, device="cuda")
    sg.sgmv_dispatch_rows(X, slots, Xs)
    for i in range(0, n, 50_000):
        for j in range(k):
            assert torch.equal(Xs[at[i:i + 50_000, j]], X[i:i + 50_000])
    Y = torch.empty_like(X)
    sg.sgmv_combine_rows(Xs, slots, Y, weights=weights)
    dYs, dw = torch.empty_like(Xs), torch.empty_like(weights)
    sg.sgmv_combine_rows_backward(X, Xs, slots, weights=weights, dYs=dYs, dweights=dw)
    h = 2.0 ** -8
    # Rows that went to the far end among them.
    look = torch.cat([torch.tensor([0, n - 1], device="cuda"), (at >= m - 4).any(1).nonzero()[:, 0]])
    x, wl = X[look].double(), weights[look].double()
    y = x * wl.sum(1, keepdim=True)                      # every copy of a row is that row
    assert ((Y[look].double() - y).abs() <= (h + 8 * u) * y.abs() + 3 * u * y.abs()).all()
    for j in range(k):
        want = x * wl[:, j, None]
        assert ((dYs[at[look, j]].double() - want).abs() <= (h + 2 * u) * want.abs()).all()
        assert ((dw[look, j].double() - (x * x).sum(1)).abs() <= (w // 64 + 32) * u * (x * x).sum(1)).all()


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_layer(act):
    n, f = 262_500, 8200
    assert n * f > 2 ** 31
    look = rows_to_look_at(n, f)
    c = lr.Layer(5, "bf16", len(look), 16, f, 8, 1, "none", 1, None, False)
    X, dY = random(6, n, 16), random(7, n, f)
    e = ta.Extra(c)
    R = random(8, n, f)
    c.X, e.residual = X[look], R[look]
    problem = sg.make_problem("bf16", n, 16, f, 8, 1, 0, 0)
    Z = torch.empty_like(R)
    W = c.proj[0]["W"]
    ws = sg.new_layer_workspace(problem, sg.SGMV_DENSE_ACT_FORWARD)
    sg.sgmv_dense_act_lora_apply(problem, X, W, (None, None, R), None, None, ws, act=ta.ACTS[act], bias=e.bias, residual=R, Z=Z)
    for got, r, what in zip((R[look], Z[look]), ta.ref(c, act, e), "YZ"):
        lr.check(got, *r, c.dtype, what)
    del R, ws
    dX, db = torch.empty_like(X), torch.empty_like(e.bias)
    ws = sg.new_layer_workspace(problem, sg.SGMV_DENSE_ACT_BACKWARD)
    sg.sgmv_dense_act_lora_backward(problem, X, W, (None, None), dY, None, None, ws, act=ta.ACTS[act], Z=Z, dX=dX, dbias=db)
    c.dY, c.proj[0]["G"] = dY[look], Z[look]
    # (The whole batch's rounding of dZ, not the few rows': a batch this large keeps no halves.)
    dz, raw, _ = ta.slopes(c, act)
    ez = raw + (lr.half_step(c.dtype) * dz.abs() if act != "none" else 0)
    lr.check(dX[look], *lr.backward(c, c.proj[0], dz, ez)[0], c.dtype, "dX")
    s, bound = torch.zeros(f, dtype=torch.float64, device="cuda"), torch.zeros(f, dtype=torch.float64, device="cuda")
    for i in range(0, n, 10_000):
        c.dY, c.proj[0]["G"], c.n = dY[i:i + 10_000], Z[i:i + 10_000], min(10_000, n - i)
        dz, raw, _ = ta.slopes(c, act)
        s += dz.sum(0)
        bound += raw.sum(0) + (n // 256 + 64) * u * dz.abs().sum(0)
    lr.check(db, s, bound, c.dtype, "dbias")
