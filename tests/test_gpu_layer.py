"""GPU parity of the layer entry points (sgmv_dense_lora_apply, sgmv_gated_lora_apply and their
backward passes) against a 64-bit reference, element by element within bounds derived
from the roundings that the header documents (tests/layer_reference.py).

Cases: one row to some thousands, sizes off every tile's multiple, every rank, both formats, segments
that are single rows, ragged, empty, repeated, absent or short of the last rows; mixed ranks (zero among them) and scales;
gradients against the formulas and against differences; graph capture, streams, accumulation, and values at
the edges of the formats."""
import numpy as np
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests import layer_reference as lr

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(list(a) or [0], dtype=torch.int32, device="cuda")


class Call:
    """The library's side of one case: tables, problem, outputs filled with NaN, a workspace of junk."""

    def __init__(self, c, op, dtype):
        self.c, self.op = c, op
        lens = np.diff(c.seg)
        self.problem = sg.make_problem(dtype, c.n, c.h_in, c.h_out, c.rank, c.P, len(c.ids), int(lens.max()) if len(lens) else 0)
        self.seg, self.ids = i32(c.seg), i32(c.ids)
        self.ws = sg.new_layer_workspace(self.problem, op)
        if self.ws.numel():
            self.ws.fill_(0xFF)         # NaN in every format: whatever is read must have been written
        self.tables = []
        for p in c.proj:
            a = sg.pointer_list([t if t.numel() else None for t in p["A"]])
            b = sg.pointer_list([t if t.numel() else None for t in p["B"]])
            ranks = i32(p["ranks"]) if p["ranks"] is not None else None
            self.tables.append((a, b, ranks, p["scales"]))

    def nan(self, *shape):
        return torch.full(shape, float("nan"), dtype=self.c.dtype, device="cuda")

    def projection(self, i, Y):
        a, b, ranks, scales = self.tables[i]
        return (a, b, Y, ranks, scales)

    def grads(self, train_w=True, fill=None):
        """Per projection: dW, lists dA, dB, and the tuple the call takes."""
        out = []
        for p in self.c.proj:
            new = (lambda t: torch.full_like(t, float("nan"))) if fill is None else (lambda t: torch.full_like(t, fill))
            dW = new(p["W"]) if train_w else None
            dA, dB = [new(t) for t in p["A"]], [new(t) for t in p["B"]]
            table = lambda ts: sg.pointer_list([t if t.numel() else None for t in ts])  # noqa: E731
            out.append((dW, dA, dB, (dW, table(dA), table(dB))))
        return out


def run_dense(c, dtype):
    call = Call(c, sg.SGMV_DENSE_FORWARD, dtype)
    Y = call.nan(c.n, c.h_out)
    sg.sgmv_dense_lora_apply(call.problem, c.X, c.proj[0]["W"], call.projection(0, Y), call.seg, call.ids, call.ws)
    return Y


def run_gated(c, dtype, act, keep=True):
    call = Call(c, sg.SGMV_GATED_FORWARD, dtype)
    H, G, U_ = (call.nan(c.n, c.h_out) for _ in range(3))
    sg.sgmv_gated_lora_apply(call.problem, c.X, c.proj[0]["W"], c.proj[1]["W"], call.projection(0, G if keep else None),
                             call.projection(1, U_ if keep else None), H, call.seg, call.ids, call.ws, act=act)
    return H, G, U_


def run_dense_back(c, dtype, train_w=True, accumulate=False, fill=None):
    call = Call(c, sg.SGMV_DENSE_BACKWARD, dtype)
    dX, grads = call.nan(c.n, c.h_in), call.grads(train_w, fill)
    sg.sgmv_dense_lora_backward(call.problem, c.X, c.proj[0]["W"], call.projection(0, None), c.dY, call.seg, call.ids,
                                call.ws, dX=dX, grad=grads[0][3], accumulate=accumulate)
    return dX, grads


def run_gated_back(c, dtype, act, train_w=True, accumulate=False, fill=None):
    call = Call(c, sg.SGMV_GATED_BACKWARD, dtype)
    dX, grads = call.nan(c.n, c.h_in), call.grads(train_w, fill)
    sg.sgmv_gated_lora_backward(call.problem, c.X, c.proj[0]["W"], c.proj[1]["W"], call.projection(0, c.proj[0]["G"]),
                                call.projection(1, c.proj[1]["G"]), c.dY, call.seg, call.ids, call.ws, dX=dX,
                                gate_grad=grads[0][3], up_grad=grads[1][3], accumulate=accumulate, act=act)
    return dX, grads


def check_grads(c, grads, refs, train_w=True):
    for i, ((dW, dA, dB, _), (_, rA, rB, rW)) in enumerate(zip(grads, refs)):
        for k in range(c.P):
            lr.check(dA[k], *rA[k], c.dtype, f"dA[{i}][{k}]")
            lr.check(dB[k], *rB[k], c.dtype, f"dB[{i}][{k}]")
        if train_w:
            lr.check(dW, *rW, c.dtype, f"dW[{i}]")


# seed, dtype, n, h_in, h_out, rank, P, layout, ranks, scales
CASES = {
    "one_row_r8": (1, "f16", 1, 264, 136, 8, 3, "one", None, False),
    "smallest": (2, "bf16", 1, 8, 8, 16, 1, "one", None, True),
    "two_rows_r64": (3, "bf16", 2, 72, 520, 64, 2, "distinct", None, False),
    "no_lora": (4, "f16", 19, 200, 88, 16, 2, "none", None, False),
    "uncovered": (5, "bf16", 33, 520, 264, 32, 4, "uncovered", None, True),
    "distinct_r16": (6, "f16", 65, 136, 392, 16, 65, "distinct", None, False),
    "mixed_r32": (7, "f16", 129, 264, 1032, 32, 5, "mixed", None, True),
    "many_empty": (8, "bf16", 97, 136, 136, 16, 9, "many_empty", None, False),
    "ranks": (9, "f16", 150, 328, 264, 64, 6, "mixed", (8, 64, 0, 32, 16), True),
    "ranks_one_row_each": (10, "bf16", 40, 136, 328, 32, 7, "distinct", (0, 8, 24, 32), True),
    "several_tiles": (11, "bf16", 300, 1000, 1048, 16, 3, "mixed", None, False),
    "uncovered_r64": (12, "f16", 257, 72, 1376, 64, 3, "uncovered", None, False),
    "deep": (13, "bf16", 48, 4104, 72, 16, 4, "mixed", None, False),
    "wide": (14, "f16", 48, 72, 4104, 8, 4, "mixed", None, True),
}


def case(name, projections):
    seed, dtype, n, h_in, h_out, rank, P, layout, ranks, scales = CASES[name]
    return lr.Layer(seed, dtype, n, h_in, h_out, rank, P, layout, projections, ranks, scales), dtype


@pytest.mark.parametrize("name", sorted(CASES))
def test_dense_forward(name):
    c, dtype = case(name, 1)
    lr.check(run_dense(c, dtype), *lr.project(c, c.proj[0]), c.dtype, name)


@pytest.mark.parametrize("act", [sg.SGMV_ACT_SILU, sg.SGMV_ACT_GELU_TANH])
@pytest.mark.parametrize("name", sorted(CASES))
def test_gated_forward(name, act):
    c, dtype = case(name, 2)
    got = run_gated(c, dtype, act)
    for g, (ref, bound), what in zip(got, lr.gate(c, act), "HGU"):
        lr.check(g, ref, bound, c.dtype, f"{name} {what}", rounded=True)
    assert torch.equal(run_gated(c, dtype, act, keep=False)[0], got[0])  # G and U are optional


@pytest.mark.parametrize("name", sorted(CASES))
def test_dense_backward(name):
    c, dtype = case(name, 1)
    dX, grads = run_dense_back(c, dtype)
    d = c.dY.double()
    ref = lr.backward(c, c.proj[0], d, torch.zeros_like(d))
    lr.check(dX, *ref[0], c.dtype, f"{name} dX")
    check_grads(c, grads, [ref])


@pytest.mark.parametrize("act", [sg.SGMV_ACT_SILU, sg.SGMV_ACT_GELU_TANH])
@pytest.mark.parametrize("name", sorted(CASES))
def test_gated_backward(name, act):
    c, dtype = case(name, 2)
    dX, grads = run_gated_back(c, dtype, act)
    refs = [lr.backward(c, p, *d) for p, d in zip(c.proj, lr.gate_backward(c, act))]
    lr.check(dX, refs[0][0][0] + refs[1][0][0], refs[0][0][1] + refs[1][0][1], c.dtype, f"{name} dX")
    check_grads(c, grads, refs)


# Sizes that reach the largest tiles, whole rounds of them, splits of the contraction and of the rows.
LARGE = {
    "tile256": (21, "bf16", 2055, 1032, 4360, 16, 5, "mixed", None, True),
    "tile256_r64": (22, "f16", 4096, 264, 4096, 64, 4, "mixed", None, False),
    "split_deep": (23, "bf16", 520, 8200, 520, 32, 3, "uncovered", None, False),
    "distinct_wide": (24, "f16", 700, 264, 2056, 16, 40, "distinct", None, False),
    "one_long_segment": (25, "bf16", 3000, 136, 1032, 8, 1, "one", None, False),
    "tile192_out": (27, "f16", 190, 72, 33000, 64, 3, "uncovered", (64, 8, 32), True),
    "tile192_in": (28, "bf16", 181, 33000, 72, 16, 3, "mixed", None, False),
    "few_rows_term_in_tile": (29, "f16", 20, 1160, 264, 64, 3, "uncovered", (64, 8, 24), True),
    "few_rows_one_segment": (30, "bf16", 60, 2056, 136, 32, 2, "one", None, False),
    "hundred_rows_r64": (31, "f16", 100, 1032, 4104, 64, 4, "mixed", None, True),
    "hundred_rows_term_in_tile": (32, "bf16", 100, 136, 11016, 64, 2, "one", None, True),
    "forty_rows_term_in_tile": (33, "f16", 40, 72, 24008, 64, 2, "one", None, False),
    "many_loras_few_segments": (26, "f16", 1500, 264, 520, 32, 60, "uncovered", (32, 8, 16), True),
}


@pytest.mark.parametrize("name", sorted(LARGE))
def test_large(name):
    seed, dtype, n, h_in, h_out, rank, P, layout, ranks, scales = LARGE[name]
    c = lr.Layer(seed, dtype, n, h_in, h_out, rank, P, layout, 2, ranks, scales)
    lr.check(run_dense(c, dtype), *lr.project(c, c.proj[0]), c.dtype, f"{name} Y")
    for g, (ref, bound), what in zip(run_gated(c, dtype, 0), lr.gate(c, 0), "HGU"):
        lr.check(g, ref, bound, c.dtype, f"{name} {what}", rounded=True)
    dX, grads = run_gated_back(c, dtype, 0)
    refs = [lr.backward(c, p, *d) for p, d in zip(c.proj, lr.gate_backward(c, 0))]
    lr.check(dX, refs[0][0][0] + refs[1][0][0], refs[0][0][1] + refs[1][0][1], c.dtype, f"{name} dX")
    check_grads(c, grads, refs)
    dX, grads = run_dense_back(c, dtype)
    d = c.dY.double()
    ref = lr.backward(c, c.proj[0], d, torch.zeros_like(d))
    lr.check(dX, *ref[0], c.dtype, f"{name} dense dX")
    check_grads(c, grads, [ref])


@pytest.mark.parametrize("train_w", [True, False])
@pytest.mark.parametrize("name", ["mixed_r32", "uncovered", "ranks", "no_lora"])
def test_accumulate_adds_and_leaves_unused_loras(name, train_w):
    """accumulate=1: the gradient on top of what is there (2.0), rounded once; LoRAs without rows untouched."""
    c, dtype = case(name, 2)
    _, grads = run_gated_back(c, dtype, 0, train_w=train_w, accumulate=True, fill=2.0)
    refs = [lr.backward(c, p, *d) for p, d in zip(c.proj, lr.gate_backward(c, 0))]
    used = {k for lo, hi, k in c.pieces}
    for i, ((dW, dA, dB, _), (_, rA, rB, rW)) in enumerate(zip(grads, refs)):
        for k in range(c.P):
            for got, (ref, bound), what in ((dA[k], rA[k], "dA"), (dB[k], rB[k], "dB")):
                if k not in used:
                    assert (got == 2.0).all()
                else:
                    lr.check(got, ref + 2.0, bound + lr.U * (ref.abs() + 2.0), c.dtype, f"{what}[{i}][{k}]")
        if train_w:
            lr.check(dW, rW[0] + 2.0, rW[1] + lr.U * (rW[0].abs() + 2.0), c.dtype, f"dW[{i}]")


def test_backward_parts_are_optional():
    """Each wanted part alone equals the same part of the whole call, bit for bit; null table entries are skipped."""
    c, dtype = case("mixed_r32", 2)
    dX, grads = run_gated_back(c, dtype, 0)
    call = Call(c, sg.SGMV_GATED_BACKWARD, dtype)
    W = [p["W"] for p in c.proj]

    def run(dX=None, g=None, u=None):
        sg.sgmv_gated_lora_backward(call.problem, c.X, W[0], W[1], call.projection(0, c.proj[0]["G"]),
                                    call.projection(1, c.proj[1]["G"]), c.dY, call.seg, call.ids, call.ws, dX=dX,
                                    gate_grad=g, up_grad=u)

    alone = call.nan(c.n, c.h_in)
    run(dX=alone)
    assert torch.equal(alone, dX)
    for i in range(2):
        new = call.grads()[i]
        parts = [(new[3][0], None, None), (None, new[3][1], None), (None, None, new[3][2])]
        for part in parts:
            run(**{"gu"[i]: part})
        assert torch.equal(new[0], grads[i][0])
        assert all(torch.equal(a, b) for a, b in zip(new[1] + new[2], grads[i][1] + grads[i][2]))
    used = c.pieces[0][2]
    keep = torch.full_like(c.proj[0]["A"][used], 7.0)
    table = [torch.empty_like(t) for t in c.proj[0]["A"]]
    ptrs = sg.pointer_list([None if k == used else t for k, t in enumerate(table)])
    run(g=(None, ptrs, None))
    torch.cuda.synchronize()
    assert (keep == 7.0).all()
    assert all(torch.equal(t, grads[0][1][k]) for k, t in enumerate(table) if k != used)


def test_no_rows_writes_zero_gradients():
    c = lr.Layer(31, "f16", 0, 136, 72, 16, 3, "none", 1, None, False)
    dX, grads = run_dense_back(c, "f16")
    dW, dA, dB, _ = grads[0]
    assert (dW == 0).all() and all((t == 0).all() for t in dA + dB)
    _, grads = run_dense_back(c, "f16", accumulate=True, fill=3.0)
    dW, dA, dB, _ = grads[0]
    assert (dW == 3).all() and all((t == 3).all() for t in dA + dB)
    assert run_dense(c, "f16").shape == (0, 72)


@pytest.mark.parametrize("act", [0, 1])
def test_gated_gradient_against_differences(act):
    """The gated backward's dX, dA and dB against central differences of the 64-bit block along random directions.
    The backward reads G and U rounded to the format (h of each), so a directional derivative may be off by the
    stored values' rounding; the bound propagates it: d(loss) / d(G or U) is known up to |second derivatives| * h * |G|."""
    c = lr.Layer(41, "f16", 24, 136, 72, 16, 2, "mixed", 2, None, True)
    H, G, U_ = run_gated(c, "f16", act)
    c.proj[0]["G"], c.proj[1]["G"] = G, U_
    dX, grads = run_gated_back(c, "f16", act)
    torch.cuda.synchronize()
    h = lr.half_step(c.dtype)

    def loss(x, a, b):
        y = []
        for i, p in enumerate(c.proj):
            out = x @ p["W"].double()
            for lo, hi, k in c.pieces:
                out[lo:hi] += lr.scale_of(p, k) * (x[lo:hi] @ a[i][k] @ b[i][k])
            y.append(out)
        return float((lr.act(act, y[0])[0] * y[1] * c.dY.double()).sum())

    x0 = c.X.double()
    a0 = [[t.double() for t in p["A"]] for p in c.proj]
    b0 = [[t.double() for t in p["B"]] for p in c.proj]
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda t: torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    refs = [lr.backward(c, p, *d) for p, d in zip(c.proj, lr.gate_backward(c, act))]
    # What rounding G and U once does to dG and dU: |act''| <= 1.2, |act'| <= 1.13.
    g, u, dh = G.double().abs(), U_.double().abs(), c.dY.double().abs()
    eg, eu = h * dh * (1.2 * u * g + 1.13 * u), h * dh * 1.13 * g
    extra = [lr.backward(c, p, torch.zeros_like(e), e) for p, e in zip(c.proj, (eg, eu))]
    eps = 1e-5
    for trial in range(3):
        vx = rand(x0)
        diff = (loss(x0 + eps * vx, a0, b0) - loss(x0 - eps * vx, a0, b0)) / (2 * eps)
        bound = sum(r[0][1] for r in refs) + sum(e[0][1] for e in extra)
        bound = ((bound + h * (dX.double().abs() + bound)) * vx.abs()).sum()
        assert abs(float((dX.double() * vx).sum()) - diff) <= float(bound) + 1e-6 * abs(diff)
        for i in range(2):
            k = c.pieces[trial % len(c.pieces)][2]
            for part, base in ((1, a0), (2, b0)):
                v = rand(base[i][k])
                plus = [[t + eps * v if (j, m) == (i, k) else t for m, t in enumerate(ts)] for j, ts in enumerate(base)]
                minus = [[t - eps * v if (j, m) == (i, k) else t for m, t in enumerate(ts)] for j, ts in enumerate(base)]
                if part == 1:
                    diff = (loss(x0, plus, b0) - loss(x0, minus, b0)) / (2 * eps)
                else:
                    diff = (loss(x0, a0, plus) - loss(x0, a0, minus)) / (2 * eps)
                got = grads[i][part][k].double()
                bound = refs[i][part][k][1] + extra[i][part][k][1]
                bound = ((bound + h * (got.abs() + bound)) * v.abs()).sum()
                assert abs(float((got * v).sum()) - diff) <= float(bound) + 1e-6 * abs(diff)


@pytest.mark.parametrize("name", ["one_row_r8", "distinct_r16", "several_tiles"])
def test_forward_then_backward_in_a_graph(name):
    """A training step's forward and backward (each with its own workspace) captured once and replayed, with eager
    calls on other buffers between the replays; every replay equals the eager result bit for bit."""
    c, dtype = case(name, 2)
    H, G, U_ = run_gated(c, dtype, 0)
    c.proj[0]["G"], c.proj[1]["G"] = G, U_
    dX, grads = run_gated_back(c, dtype, 0)
    fwd, bwd = Call(c, sg.SGMV_GATED_FORWARD, dtype), Call(c, sg.SGMV_GATED_BACKWARD, dtype)
    H2, G2, U2, dX2 = (t.clone() for t in (H, G, U_, dX))
    new = bwd.grads()
    W = [p["W"] for p in c.proj]

    def step():
        sg.sgmv_gated_lora_apply(fwd.problem, c.X, W[0], W[1], fwd.projection(0, G2), fwd.projection(1, U2), H2, fwd.seg,
                                 fwd.ids, fwd.ws)
        sg.sgmv_gated_lora_backward(bwd.problem, c.X, W[0], W[1], bwd.projection(0, G2), bwd.projection(1, U2), c.dY,
                                    bwd.seg, bwd.ids, bwd.ws, dX=dX2, gate_grad=new[0][3], up_grad=new[1][3])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (H2, G2, U2, dX2):
            t.fill_(float("nan"))
        graph.replay()
        run_dense(c, dtype)             # the program's own eager work between replays
        torch.cuda.synchronize()
        assert torch.equal(H2, H) and torch.equal(G2, G) and torch.equal(U2, U_) and torch.equal(dX2, dX)
        for a, b in zip(new, grads):
            assert torch.equal(a[0], b[0])
            assert all(torch.equal(x, y) for x, y in zip(a[1] + a[2], b[1] + b[2]))


def test_two_streams_at_once():
    """Two calls at once on two streams, each with its own workspace, equal the calls made one by one."""
    (c1, d1), (c2, d2) = case("mixed_r32", 2), case("several_tiles", 2)
    want = [run_gated(c1, d1, 0)[0], run_gated(c2, d2, 1)[0]]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = run_gated(c1, d1, 0)[0]
        with torch.cuda.stream(s2):
            b = run_gated(c2, d2, 1)[0]
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_rows_of_other_loras_do_not_reach_a_gradient():
    """NaN and infinity in one segment's rows of X and dY stay in that segment's LoRA: the others' gradients and the
    other rows of dX and Y are what they are without them."""
    c = lr.Layer(51, "bf16", 90, 136, 264, 16, 3, "none", 1, None, False)
    c.seg, c.ids = [0, 25, 58, 90], [2, 0, 1]
    Y, (dX, grads) = run_dense(c, "bf16"), run_dense_back(c, "bf16", train_w=False)
    c.X[30] = float("nan")
    c.dY[40] = float("inf")
    Y2, (dX2, grads2) = run_dense(c, "bf16"), run_dense_back(c, "bf16", train_w=False)
    rows = [i for i in range(90) if i not in (30,)]
    assert torch.equal(Y2[rows], Y[rows]) and Y2[30].isnan().all()
    rows = [i for i in range(90) if i != 40]
    assert torch.equal(dX2[rows], dX[rows])
    for k in (1, 2):
        assert torch.equal(grads2[0][1][k], grads[0][1][k]) and torch.equal(grads2[0][2][k], grads[0][2][k])
    assert grads2[0][1][0].isnan().any()


def test_fp16_intermediates_beyond_fp16():
    """X @ A_k beyond fp16's largest value: V stays fp32, so an output that fits comes out right."""
    c = lr.Layer(61, "f16", 70, 264, 136, 16, 2, "mixed", 1, None, False)
    p = c.proj[0]
    c.X.mul_(64)
    for k in range(2):
        p["A"][k].mul_(4096)            # V ~ 64 * 4096: far beyond 65504
        p["B"][k].mul_(2.0 ** -14)
    lr.check(run_dense(c, "f16"), *lr.project(c, p), c.dtype, "Y")
    dX, grads = run_dense_back(c, "f16")
    d = c.dY.double()
    ref = lr.backward(c, p, d, torch.zeros_like(d))
    lr.check(dX, *ref[0], c.dtype, "dX")
    for k in range(2):
        lr.check(grads[0][1][k], *ref[1][k], c.dtype, "dA")


@pytest.mark.parametrize("n", [40, 200, 1100])
def test_fp16_intermediates_below_fp16(n):
    """V and dV far below 1, in steps from row to row: fp32 holds them, so outputs and gradients of ordinary size
    must not lose them to fp16's denormals."""
    c = lr.Layer(63, "f16", n, 264, 136, 16, 3, "mixed", 1, None, False)
    p = c.proj[0]
    step = torch.tensor([1.0, 2.0 ** -8, 2.0 ** -5, 2.0 ** -10], device="cuda").repeat(n)[:n, None]
    c.X.mul_(step.half())
    c.dY.mul_(step.flip(0).half())
    for k in range(3):
        p["A"][k].mul_(2.0 ** -7)           # V ~ 2^-7 .. 2^-17
        p["B"][k].mul_(2.0 ** (4 - 3 * k))
    p["W"].mul_(2.0 ** -12)                 # the LoRA term is what is left to see
    p["scales"] = torch.tensor([2.0 ** 7, 2.0 ** -9, 1.0], device="cuda")
    lr.check(run_dense(c, "f16"), *lr.project(c, p), c.dtype, "Y")
    dX, grads = run_dense_back(c, "f16")
    d = c.dY.double()
    ref = lr.backward(c, p, d, torch.zeros_like(d))
    lr.check(dX, *ref[0], c.dtype, "dX")
    check_grads(c, grads, [ref])


def test_gate_far_out():
    """Gates at the ends of the format: silu and its slope go to 0 and to the identity without NaN."""
    c = lr.Layer(71, "bf16", 16, 64, 64, 8, 1, "none", 2, None, False)
    far = torch.tensor([-1e30, -300.0, -88.0, -20.0, 0.0, 20.0, 300.0, 1e30], device="cuda")
    c.proj[0]["G"] = far.repeat(16, 8).to(torch.bfloat16)
    c.dY.clamp_(-2, 2)
    for act in (0, 1):
        dX, grads = run_gated_back(c, "bf16", act)
        refs = [lr.backward(c, p, *d) for p, d in zip(c.proj, lr.gate_backward(c, act))]
        assert torch.isfinite(grads[0][0].double()).all()
        lr.check(grads[0][0], *refs[0][3], c.dtype, "dWg")


def test_rows_behind_the_last_row_are_left_alone():
    """Outputs are written up to n_rows and h_out only: guard rows around them keep their values."""
    c, dtype = case("mixed_r32", 1)
    call = Call(c, sg.SGMV_DENSE_FORWARD, dtype)
    buf = torch.full((c.n + 2, c.h_out), 5.0, dtype=c.dtype, device="cuda")
    sg.sgmv_dense_lora_apply(call.problem, c.X, c.proj[0]["W"], call.projection(0, buf[1:-1]), call.seg, call.ids, call.ws)
    assert torch.equal(buf[1:-1], run_dense(c, dtype))
    assert (buf[0] == 5).all() and (buf[-1] == 5).all()


def test_same_call_twice_is_bitwise_equal():
    for name in ("several_tiles", "ranks"):
        c, dtype = case(name, 2)
        a, b = run_gated_back(c, dtype, 0), run_gated_back(c, dtype, 0)
        assert torch.equal(a[0], b[0])
        for x, y in zip(a[1], b[1]):
            assert torch.equal(x[0], y[0]) and all(torch.equal(s, t) for s, t in zip(x[1] + x[2], y[1] + y[2]))


@pytest.mark.parametrize("n,h_in,h_out", [(60, 136, 264), (420, 264, 520)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_broken_lora_stays_with_its_own_rows(n, h_in, h_out, bad):
    """NaN or infinity in one LoRA's matrices reaches that LoRA's rows only, where the tiles add the term and where
    the epilogue does, and dX likewise."""
    c = lr.Layer(81, "bf16", n, h_in, h_out, 16, 3, "none", 2, None, False)
    c.seg, c.ids = [0, n // 3 + 1, n // 2 + 3, n], [0, 2, 1]
    before = run_gated(c, "bf16", 0), run_gated_back(c, "bf16", 0, train_w=False)[0], run_dense(c, "bf16")
    for p in c.proj:
        p["A"][2][5] = bad
        p["B"][2][3, 7] = bad
    after = run_gated(c, "bf16", 0), run_gated_back(c, "bf16", 0, train_w=False)[0], run_dense(c, "bf16")
    mine = slice(c.seg[1], c.seg[2])
    others = [i for i in range(n) if not c.seg[1] <= i < c.seg[2]]
    for a, b in list(zip(before[0], after[0])) + [(before[1], after[1]), (before[2], after[2])]:
        assert torch.equal(a[others], b[others])
        assert not torch.isfinite(b[mine]).all()


@pytest.mark.parametrize("wide", ["in", "out"])
def test_offsets_beyond_32_bits(wide):
    """X (or dY) of more than 2^31 elements, zero but for the last rows: outputs of those rows and the gradients,
    which only they reach, against 64 bits on those rows alone."""
    big, tail = 4104, 700
    n = 2 ** 31 // big + 2000
    h_in, h_out = (big, 24) if wide == "in" else (24, big)
    c = lr.Layer(91, "bf16", tail, h_in, h_out, 8, 2, "none", 1, None, False)
    small = lr.Layer(91, "bf16", tail, h_in, h_out, 8, 2, "none", 1, None, False)
    c.n = n
    for name, width in (("X", h_in), ("dY", h_out)):
        full = torch.zeros(n, width, dtype=c.dtype, device="cuda")
        full[-tail:] = getattr(small, name)
        setattr(c, name, full)
    c.seg, c.ids = [0, n - 300, n], [0, 1]
    small.seg, small.ids = [0, tail - 300, tail], [0, 1]
    Y = run_dense(c, "bf16")
    lr.check(Y[-tail:], *lr.project(small, small.proj[0]), c.dtype, "Y")
    assert (Y[:-tail] == 0).all()
    del Y
    dX, grads = run_dense_back(c, "bf16")
    d = small.dY.double()
    small.n = n  # the bounds count every row that is summed
    ref = lr.backward(small, small.proj[0], d, torch.zeros_like(d))
    lr.check(dX[-tail:], *ref[0], c.dtype, "dX")
    check_grads(c, grads, [ref])


def test_binding_refuses_wrong_shapes():
    c, dtype = case("mixed_r32", 1)
    call = Call(c, sg.SGMV_DENSE_FORWARD, dtype)
    Y = call.nan(c.n, c.h_out)
    good = dict(X=c.X, W=c.proj[0]["W"], proj=call.projection(0, Y), seg=call.seg, ids=call.ids, ws=call.ws)

    def run(**kw):
        a = {**good, **kw}
        sg.sgmv_dense_lora_apply(call.problem, a["X"], a["W"], a["proj"], a["seg"], a["ids"], a["ws"])

    run()
    A, B, Yp, ranks, scales = good["proj"]
    for kw in (dict(X=c.X[:-1]), dict(W=c.proj[0]["W"].t()), dict(W=c.proj[0]["W"].float()), dict(X=c.X.cpu()),
               dict(proj=(A[:-1], B, Yp, ranks, scales)), dict(proj=(A, B[:1], Yp, ranks, scales)),
               dict(proj=(A, B, Yp[:, :8], ranks, scales)), dict(proj=(A, B, Yp, ranks, scales[:-1])),
               dict(proj=(A, B, Yp, call.ids[:1], scales)), dict(seg=call.seg[:-1]), dict(ids=call.ids[:-1]),
               dict(seg=call.seg.long())):
        with pytest.raises(ValueError):
            run(**kw)
    with pytest.raises(sg.SgmvError):
        run(ws=call.ws[:-16])
