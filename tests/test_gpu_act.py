"""GPU parity of the layer with bias, activation and residual and of its gradients, against 64 bits within derived bounds (those of
tests/layer_reference.py for the products).

The epilogue adds, with u = 2^-24: one rounding each of z + bias and act + residual; the logistic function of x, by exponential and
reciprocal, is off by (|x| + 8) 2^-23 of itself (the argument's rounding times log2 e and some units in the last place), gelu's x
by another 3 u of itself; erfc(x) by (2 x^2 + 20) 2^-23 of itself (16 units in the last place, and the argument's rounding times
the logarithmic derivative, at most 2 |x| + 1).  Values below 2^-120 may be flushed.  |act'| <= 1.13 for every activation."""
import math

import numpy as np
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests import layer_reference as lr
from tests.test_gpu_layer import CASES, LARGE, Call, case, check_grads, run_dense, run_dense_back

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
ACTS = {"none": sg.SGMV_ACT_NONE, "relu": sg.SGMV_ACT_RELU, "silu": sg.SGMV_ACT_SILU, "gelu_tanh": sg.SGMV_ACT_GELU_TANH,
        "gelu": sg.SGMV_ACT_GELU}


def act64(kind, z):
    """Value, derivative and the bound of the fp32 value's error."""
    if kind == "none":
        return z, torch.ones_like(z), torch.zeros_like(z)
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double(), torch.zeros_like(z)
    if kind == "gelu":
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), (z * phi).abs() * (z * z + 24) * 2 * u + 2.0 ** -120
    value, slope = lr.act(ACTS[kind], z)
    x = z if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    return value, slope, value.abs() * (4 * x.abs() + 20) * u + 2.0 ** -120


class Extra:
    """Bias and residual beside a layer's case; rows of z far on both sides of 0 among the ordinary ones."""

    def __init__(self, c, seed=0, bias=True, residual=True):
        g = torch.Generator().manual_seed(seed + 900)
        self.bias = (torch.randn(c.h_out, generator=g) * 2).to(c.dtype).cuda() if bias else None
        self.residual = torch.randn(c.n, c.h_out, generator=g).to(c.dtype).cuda() if residual else None


def run(c, dtype, act, e, keep=True, Y=None):
    call = Call(c, sg.SGMV_DENSE_ACT_FORWARD, dtype)
    Y = call.nan(c.n, c.h_out) if Y is None else Y
    Z = call.nan(c.n, c.h_out) if keep else None
    sg.sgmv_dense_act_lora_apply(call.problem, c.X, c.proj[0]["W"], call.projection(0, Y), call.seg, call.ids, call.ws,
                                 act=ACTS[act], bias=e.bias, residual=e.residual, Z=Z)
    return Y, Z


def run_back(c, dtype, act, train_w=True, accumulate=False, fill=None, dbias=True):
    call = Call(c, sg.SGMV_DENSE_ACT_BACKWARD, dtype)
    dX, grads = call.nan(c.n, c.h_in), call.grads(train_w, fill)
    db = torch.full((c.h_out,), float("nan") if fill is None else fill, dtype=c.dtype, device="cuda") if dbias else None
    sg.sgmv_dense_act_lora_backward(call.problem, c.X, c.proj[0]["W"], call.projection(0, None), c.dY, call.seg, call.ids, call.ws,
                                    act=ACTS[act], Z=c.proj[0]["G"] if act != "none" else None, dX=dX, grad=grads[0][3],
                                    dbias=db, accumulate=accumulate)
    return dX, grads, db


def ref(c, act, e):
    z, ez = lr.project(c, c.proj[0])
    if e.bias is not None:
        z = z + e.bias.double()
        ez = ez + 2 * u * (z.abs() + ez)
    y, _, ea = act64(act, z)
    ey = 1.13 * ez + ea
    if e.residual is not None:
        y = y + e.residual.double()
        ey = ey + 2 * u * (y.abs() + ey)
    return (y, ey), (z, ez)


def slopes(c, act):
    """dZ in 64 bits with the bounds of the unrounded value and of the one that the products take."""
    dy = c.dY.double()
    if act == "none":
        return dy, torch.zeros_like(dy), torch.zeros_like(dy)
    z = c.proj[0]["G"].double()
    dz = dy * act64(act, z)[1]
    raw = (2.0 ** -20 * dy.abs() * 1.13 * (1 + z.abs()) if act != "relu" else torch.zeros_like(dz)) + 2 * u * dz.abs()
    h = lr.half_step(c.dtype)
    if c.n <= 128 and c.n * c.h_out <= 2 ** 18:
        h = h * h
    floor = 2.0 ** -32 * 1.13 * dy.abs().amax(1, keepdim=True) if c.dtype == torch.float16 else 2.0 ** -134
    return dz, raw, raw + h * dz.abs() + floor


def check_back(c, act, got, train_w=True, old=0.0, name=""):
    dX, grads, db = got
    dz, raw, ez = slopes(c, act)
    want = lr.backward(c, c.proj[0], dz, ez, train_w)
    lr.check(dX, *want[0], c.dtype, f"{name} dX")
    if old == 0.0:
        check_grads(c, grads, [want], train_w)
    s = dz.sum(0) + old
    lr.check(db, s, raw.sum(0) + (c.n + 64) * u * (dz.abs().sum(0) + old), c.dtype, f"{name} dbias")
    return want


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("name", sorted(CASES))
def test_forward(name, act):
    c, dtype = case(name, 1)
    e = Extra(c)
    got = run(c, dtype, act, e)
    for g, r, what in zip(got, ref(c, act, e), "YZ"):
        lr.check(g, *r, c.dtype, f"{name} {what}")
    assert torch.equal(run(c, dtype, act, e, keep=False)[0], got[0])


@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("name", ["one_row_r8", "uncovered", "several_tiles"])
def test_parts_of_the_epilogue(name, bias, residual):
    c, dtype = case(name, 1)
    e = Extra(c, 1, bias, residual)
    for g, r, what in zip(run(c, dtype, "gelu_tanh", e), ref(c, "gelu_tanh", e), "YZ"):
        lr.check(g, *r, c.dtype, f"{name} {what}")
    Y, Z = run(c, dtype, "none", e)
    if not residual:
        assert torch.equal(Y, Z)
    if not bias and not residual:
        assert torch.equal(Y, run_dense(c, dtype))      # the layer's call without an epilogue


@pytest.mark.parametrize("name", ["one_row_r8", "mixed_r32", "ranks", "several_tiles"])
def test_residual_in_place(name):
    c, dtype = case(name, 1)
    e = Extra(c, 2)
    want = run(c, dtype, "silu", e)[0]
    Y = e.residual
    e.residual = Y
    assert torch.equal(run(c, dtype, "silu", e, Y=Y)[0], want)


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("name", sorted(CASES))
def test_backward(name, act):
    c, dtype = case(name, 1)
    check_back(c, act, run_back(c, dtype, act), name=name)


@pytest.mark.parametrize("name", sorted(LARGE))
def test_large(name):
    """The largest tiles, whole rounds of them, splits of the contraction and of the rows."""
    seed, dtype, n, h_in, h_out, rank, P, layout, ranks, scales = LARGE[name]
    c = lr.Layer(seed, dtype, n, h_in, h_out, rank, P, layout, 1, ranks, scales)
    act = sorted(ACTS)[seed % 5]
    e = Extra(c)
    for g, r, what in zip(run(c, dtype, act, e), ref(c, act, e), "YZ"):
        lr.check(g, *r, c.dtype, f"{name} {what}")
    check_back(c, act, run_back(c, dtype, act), name=name)


# Each tile shape writing its outputs itself (no splits, no LoRA term left over) at edges inside the tile's rows and columns.
@pytest.mark.parametrize("n,h_in,h_out", [(2300, 256, 4424), (300, 136, 16904), (500, 520, 2056), (50, 72, 33000), (20, 64, 40008)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_tiles(n, h_in, h_out, dtype):
    c = lr.Layer(n, dtype, n, h_in, h_out, 8, 1, "none", 1, None, False)
    e = Extra(c)
    for act in ("gelu_tanh", "none"):
        for g, r, what in zip(run(c, dtype, act, e), ref(c, act, e), "YZ"):
            lr.check(g, *r, c.dtype, f"{n} {what}")


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("name", ["mixed_r32", "uncovered", "no_lora"])
def test_accumulate(name, act):
    c, dtype = case(name, 1)
    got = run_back(c, dtype, act, accumulate=True, fill=2.0)
    want = check_back(c, act, got, old=2.0, name=name)
    used = {k for _, _, k in c.pieces}
    _, grads, _ = got
    for k in range(c.P):
        for g, (r, b) in ((grads[0][1][k], want[1][k]), (grads[0][2][k], want[2][k])):
            if k in used:
                lr.check(g, r + 2.0, b + lr.U * (r.abs() + 2.0), c.dtype, "gradient")
            else:
                assert (g == 2.0).all()
    lr.check(grads[0][0], want[3][0] + 2.0, want[3][1] + lr.U * (want[3][0].abs() + 2.0), c.dtype, "dW")


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_parts_of_the_backward(act):
    """Each wanted part alone equals the same part of the whole call, bit for bit; without an activation the gradients are
    those of the plain layer."""
    c, dtype = case("mixed_r32", 1)
    dX, grads, db = run_back(c, dtype, act)
    call = Call(c, sg.SGMV_DENSE_ACT_BACKWARD, dtype)

    def alone(**kw):
        call.ws.fill_(0xFF)
        sg.sgmv_dense_act_lora_backward(call.problem, c.X, c.proj[0]["W"], call.projection(0, None), c.dY, call.seg, call.ids,
                                        call.ws, act=ACTS[act], Z=c.proj[0]["G"], **kw)

    t = torch.full_like(dX, float("nan"))
    alone(dX=t)
    assert torch.equal(t, dX)
    t = torch.full_like(db, float("nan"))
    alone(dbias=t)
    assert torch.equal(t, db)
    new = call.grads()[0]
    for part in ((new[3][0], None, None), (None, new[3][1], None), (None, None, new[3][2])):
        alone(grad=part)
    assert torch.equal(new[0], grads[0][0]) and all(torch.equal(a, b) for a, b in zip(new[1] + new[2], grads[0][1] + grads[0][2]))
    if act == "none":
        dX2, plain = run_dense_back(c, dtype)
        assert torch.equal(dX2, dX) and all(torch.equal(a, b) for a, b in zip(plain[0][1], grads[0][1]))


@pytest.mark.parametrize("accumulate", [False, True])
def test_no_rows(accumulate):
    c = lr.Layer(31, "f16", 0, 136, 72, 16, 3, "none", 1, None, False)
    for act in ("none", "silu"):
        _, grads, db = run_back(c, "f16", act, accumulate=accumulate, fill=3.0)
        want = 3.0 if accumulate else 0.0
        assert (db == want).all() and (grads[0][0] == want).all() and all((t == want).all() for t in grads[0][1] + grads[0][2])
    assert run(c, "f16", "silu", Extra(c))[0].shape == (0, 72)


@pytest.mark.parametrize("act", sorted(set(ACTS) - {"none"}))
def test_values_at_the_edges(act):
    """z at 0, far out on both sides and not finite: values and slopes by the formulas, and a row's NaN stays in the row."""
    n, f = 9, 64
    c = lr.Layer(71, "bf16", n, 8, f, 8, 1, "none", 1, None, False)
    c.X.zero_()
    e = Extra(c, residual=False)
    grid = torch.cat([torch.tensor([0.0, -0.0, 1e-30, -1e-30, 30.0, -30.0, 1e4, -1e4]), torch.linspace(-12, 12, f - 8)])
    e.bias = grid.to(c.dtype).cuda()
    Y, Z = run(c, "bf16", act, e)
    z = e.bias.double().expand(n, f)
    y, slope, ea = act64(act, z)
    lr.check(Z, z, torch.zeros_like(z), c.dtype, "Z")
    lr.check(Y, y, ea, c.dtype, "Y")
    assert torch.isfinite(Y.float()).all() and (Y[:, :2] == 0).all()
    c.proj[0]["G"] = Z
    check_back(c, act, run_back(c, "bf16", act))
    c.X[4] = float("nan")
    Y2, _ = run(c, "bf16", act, e)
    rows = [i for i in range(n) if i != 4]
    assert torch.equal(Y2[rows], Y[rows]) and Y2[4].isnan().all()


@pytest.mark.parametrize("n", [20, 300])
@pytest.mark.parametrize("ratio", [1.0, 2.0 ** -18])
def test_fp16_rows_of_small_gradients(n, ratio):
    """dY of fp16's smallest numbers, and rows 2^18 apart: dZ keeps a power of two per row, so no row loses its bits."""
    c, _ = lr.Layer(81, "f16", n, 136, 264, 16, 3, "mixed", 1, None, False), None
    step = torch.where(torch.arange(n) % 2 == 0, 2.0 ** -6, 2.0 ** -6 * ratio)[:, None].cuda().half()
    c.dY.mul_(step)
    check_back(c, "gelu_tanh", run_back(c, "f16", "gelu_tanh"))


@pytest.mark.parametrize("n,h_out", [(5, 2048), (9, 2056), (150, 4096), (40, 4104), (131, 8192), (7, 8200), (133, 16384), (6, 16392), (140, 20008)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_widths_of_the_activation_backward(n, h_out, dtype):
    """Either side of every width that changes how a row of dZ is shared out, with rows of zeros and of tiny values among them."""
    c = lr.Layer(n, dtype, n, 16, h_out, 8, 2, "one", 1, None, False)
    c.dY[1] = 0
    c.dY[2] *= 2.0 ** -12
    check_back(c, "silu", run_back(c, dtype, "silu"))


@pytest.mark.parametrize("act", sorted(set(ACTS) - {"relu"}))
def test_gradient_against_differences(act):
    """dX, dA, dB and dbias against central differences of the 64-bit layer along random directions; the backward reads Z rounded
    once (h |z|), which moves act' by |act''| <= 1.2 of that.  (relu has no second derivative at 0; its slope is checked above.)"""
    c = lr.Layer(41, "f16", 24, 136, 72, 16, 2, "mixed", 1, None, True)
    p, e = c.proj[0], Extra(c)
    _, Z = run(c, "f16", act, e)
    p["G"] = Z
    dX, grads, db = run_back(c, "f16", act)
    h = lr.half_step(c.dtype)

    def loss(x, a, b, bias):
        z = x @ p["W"].double() + bias
        for lo, hi, k in c.pieces:
            z[lo:hi] += lr.scale_of(p, k) * (x[lo:hi] @ a[k] @ b[k])
        return float((act64(act, z)[0] * c.dY.double()).sum())

    base = [c.X.double(), [t.double() for t in p["A"]], [t.double() for t in p["B"]], e.bias.double()]
    dz, raw, ez = slopes(c, act)
    extra = 1.2 * h * Z.double().abs() * c.dY.double().abs() if act != "none" else torch.zeros_like(dz)
    want, moved = lr.backward(c, p, dz, ez), lr.backward(c, p, torch.zeros_like(dz), extra)
    gen = torch.Generator(device="cuda").manual_seed(5)
    eps = 1e-5

    def compare(index, k, got, bound):
        t = base[index] if k is None else base[index][k]
        v = torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64)

        def at(s):
            args = list(base)
            args[index] = t + s * v if k is None else [x + s * v if j == k else x for j, x in enumerate(base[index])]
            return loss(*args)

        diff = (at(eps) - at(-eps)) / (2 * eps)
        full = ((bound + h * (got.double().abs() + bound)) * v.abs()).sum()
        assert abs(float((got.double() * v).sum()) - diff) <= float(full) + 1e-6 * abs(diff)

    compare(0, None, dX, want[0][1] + moved[0][1])
    for k in sorted({k for _, _, k in c.pieces}):
        compare(1, k, grads[0][1][k], want[1][k][1] + moved[1][k][1])
        compare(2, k, grads[0][2][k], want[2][k][1] + moved[2][k][1])
    compare(3, None, db, raw.sum(0) + extra.sum(0) + 100 * u * dz.abs().sum(0))


@pytest.mark.parametrize("name", ["one_row_r8", "distinct_r16", "several_tiles"])
def test_every_replay_writes_every_output(name):
    c, dtype = case(name, 1)
    e = Extra(c)
    Y, Z = run(c, dtype, "gelu", e)
    c.proj[0]["G"] = Z
    dX, grads, db = run_back(c, dtype, "gelu")
    want = [Y, Z, dX, db, grads[0][0]] + grads[0][1] + grads[0][2]
    fwd, bwd = Call(c, sg.SGMV_DENSE_ACT_FORWARD, dtype), Call(c, sg.SGMV_DENSE_ACT_BACKWARD, dtype)
    Y2, Z2, dX2, db2 = (torch.empty_like(t) for t in (Y, Z, dX, db))
    new = bwd.grads()[0]
    out = [Y2, Z2, dX2, db2, new[0]] + new[1] + new[2]

    def step():
        sg.sgmv_dense_act_lora_apply(fwd.problem, c.X, c.proj[0]["W"], fwd.projection(0, Y2), fwd.seg, fwd.ids, fwd.ws,
                                     act=ACTS["gelu"], bias=e.bias, residual=e.residual, Z=Z2)
        sg.sgmv_dense_act_lora_backward(bwd.problem, c.X, c.proj[0]["W"], bwd.projection(0, None), c.dY, bwd.seg, bwd.ids, bwd.ws,
                                        act=ACTS["gelu"], Z=Z2, dX=dX2, grad=new[3], dbias=db2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        for ws in (fwd.ws, bwd.ws):
            ws.fill_(0xFF)
        graph.replay()
        run_dense(c, dtype)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), f"output {i}"


def test_two_streams_at_once():
    (c1, d1), (c2, d2) = case("mixed_r32", 1), case("several_tiles", 1)
    e1, e2 = Extra(c1), Extra(c2)
    want = [run(c1, d1, "gelu", e1)[0], run_back(c2, d2, "silu")[0]]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = run(c1, d1, "gelu", e1)[0]
        with torch.cuda.stream(s2):
            b = run_back(c2, d2, "silu")[0]
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
