"""Gradients of a layer with an activation whose dZ is asked for as two halves (SGMV_DZ_HALVES): within the bounds of h^2 instead of
h for dZ at every size, and what small batches have by themselves bit for bit."""
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests import layer_reference as lr
from tests.test_gpu_act import ACTS, act64, run_back, u
from tests.test_gpu_act_wide import BACKWARD, layer
from tests.test_gpu_layer import CASES, LARGE, Call, case, check_grads

pytestmark = pytest.mark.gpu

OP = sg.SGMV_DENSE_ACT_BACKWARD | sg.SGMV_DZ_HALVES


def run_halves(c, dtype, act, accumulate=False, fill=None):
    call = Call(c, OP, dtype)
    dX, grads = call.nan(c.n, c.h_in), call.grads(True, fill)
    db = torch.full((c.h_out,), float("nan") if fill is None else fill, dtype=c.dtype, device="cuda")
    sg.sgmv_dense_act_lora_backward(call.problem, c.X, c.proj[0]["W"], call.projection(0, None), c.dY, call.seg, call.ids, call.ws,
                                    act=ACTS[act] | sg.SGMV_DZ_HALVES, Z=c.proj[0]["G"] if act != "none" else None, dX=dX,
                                    grad=grads[0][3], dbias=db, accumulate=accumulate)
    return dX, grads, db


def reference(c, act):
    """Gradients and bounds as in tests/test_gpu_act.py with h^2 for dZ."""
    dy = c.dY.double()
    dz, raw, ez = dy, torch.zeros_like(dy), torch.zeros_like(dy)
    if act != "none":
        z = c.proj[0]["G"].double()
        dz = dy * act64(act, z)[1]
        raw = (2.0 ** -20 * dy.abs() * 1.13 * (1 + z.abs()) if act != "relu" else torch.zeros_like(dz)) + 2 * u * dz.abs()
        floor = 2.0 ** -32 * 1.13 * dy.abs().amax(1, keepdim=True) if c.dtype == torch.float16 else 2.0 ** -134
        ez = raw + lr.half_step(c.dtype) ** 2 * dz.abs() + floor
    return lr.backward(c, c.proj[0], dz, ez), (dz.sum(0), raw.sum(0) + (c.n + 64) * u * dz.abs().sum(0))


def check(c, act, got, name):
    dX, grads, db = got
    want, bias = reference(c, act)
    lr.check(dX, *want[0], c.dtype, f"{name} dX")
    check_grads(c, grads, [want])
    lr.check(db, *bias, c.dtype, f"{name} dbias")


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("name", sorted(CASES))
def test_small(name, act):
    c, dtype = case(name, 1)
    got = run_halves(c, dtype, act)
    check(c, act, got, name)
    if act == "none" or (c.n <= 128 and c.n * c.h_out <= 2 ** 18):
        dX, grads, db = run_back(c, dtype, act)
        new = [got[0], got[2], got[1][0][0]] + got[1][0][1] + got[1][0][2]
        old = [dX, db, grads[0][0]] + grads[0][1] + grads[0][2]
        assert all(torch.equal(a, b) for a, b in zip(new, old))


@pytest.mark.parametrize("name", sorted(LARGE))
def test_large(name):
    seed, dtype, n, h_in, h_out, rank, P, layout, ranks, scales = LARGE[name]
    c = lr.Layer(seed, dtype, n, h_in, h_out, rank, P, layout, 1, ranks, scales)
    act = sorted(set(ACTS) - {"none"})[seed % 4]
    check(c, act, run_halves(c, dtype, act), name)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", BACKWARD, ids=str)
def test_sizes_of_the_wide_tiles(shape, dtype):
    c = layer(shape, dtype)
    check(c, "silu", run_halves(c, dtype, "silu"), str(shape))


@pytest.mark.parametrize("ratio", [1.0, 2.0 ** -18])
@pytest.mark.parametrize("n,h_out", [(300, 264), (140, 4104), (130, 16392)])
def test_fp16_rows_of_small_gradients(n, h_out, ratio):
    c = lr.Layer(81, "f16", n, 136, h_out, 16, 3, "mixed", 1, None, False)
    c.dY.mul_(torch.where(torch.arange(n) % 2 == 0, 2.0 ** -6, 2.0 ** -6 * ratio)[:, None].cuda().half())
    check(c, "gelu_tanh", run_halves(c, "f16", "gelu_tanh"), "small")


def test_what_it_is_for():
    """2-norms off the 64-bit gradients are those of the outputs' own rounding, uniform within half a step of each value's binade:
    step / sqrt 12 on average (of 16000 values and more, to within some percent)."""
    c = lr.Layer(5, "bf16", 2100, 1032, 1384, 16, 3, "mixed", 1, None, True)
    want, _ = reference(c, "gelu")
    got = run_halves(c, "bf16", "gelu")
    for g, (r, _) in ((got[0], want[0]), (got[1][0][0], want[3]), (got[1][0][1][0], want[1][0]), (got[1][0][2][0], want[2][0])):
        step = torch.finfo(c.dtype).eps * 2.0 ** torch.floor(torch.log2(r.abs().clamp(min=1e-30)))
        own = (step * step / 12).sum().sqrt()
        assert float((g.double() - r).norm()) <= 1.05 * float(own)


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("name", ["mixed_r32", "several_tiles", "no_lora"])
def test_accumulate(name, act):
    c, dtype = case(name, 1)
    dX, grads, db = run_halves(c, dtype, act, accumulate=True, fill=2.0)
    want, bias = reference(c, act)
    lr.check(dX, *want[0], c.dtype, "dX")
    add = lambda r, b: (r + 2.0, b + lr.U * (r.abs() + 2.0))  # noqa: E731
    lr.check(db, *add(*bias), c.dtype, "dbias")
    lr.check(grads[0][0], *add(*want[3]), c.dtype, "dW")
    used = {k for _, _, k in c.pieces}
    for k in range(c.P):
        for g, r in ((grads[0][1][k], want[1][k]), (grads[0][2][k], want[2][k])):
            if k in used:
                lr.check(g, *add(*r), c.dtype, "gradient")
            else:
                assert (g == 2.0).all()


def test_every_replay_writes_every_output():
    c, dtype = case("several_tiles", 1)
    dX, grads, db = run_halves(c, dtype, "gelu")
    want = [dX, db, grads[0][0]] + grads[0][1] + grads[0][2]
    call = Call(c, OP, dtype)
    new = call.grads()[0]
    out = [torch.empty_like(dX), torch.empty_like(db), new[0]] + new[1] + new[2]

    def step():
        sg.sgmv_dense_act_lora_backward(call.problem, c.X, c.proj[0]["W"], call.projection(0, None), c.dY, call.seg, call.ids,
                                        call.ws, act=ACTS["gelu"] | sg.SGMV_DZ_HALVES, Z=c.proj[0]["G"], dX=out[0], grad=new[3],
                                        dbias=out[1])

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
        call.ws.fill_(0xFF)
        graph.replay()
        run_back(c, dtype, "gelu")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
