"""fp16 layers whose rows differ widely in magnitude: what one row has must not cost another row its bits.

The bounds are those of tests/layer_reference.py with every row's own floor: V and dV are held as hi + lo halves in
a unit of the row's own, so a row's value is off by h^2 of itself plus 2^-25 of that unit, whatever the other rows hold."""
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests import layer_reference as lr
from tests.test_gpu_layer import run_dense_back, run_gated_back

pytestmark = pytest.mark.gpu


def lora_gradients(c, p, d, ed):
    """(dA_k), (dB_k) as (value, bound of the unrounded sum) pairs, from the output gradient d known up to ed."""
    h, X = lr.half_step(c.dtype), c.X.double()
    out = [[[torch.zeros_like(t, dtype=torch.float64) for t in p[name]] for _ in range(2)] for name in "AB"]
    (dA, eA), (dB, eB) = out
    n = (2 * c.n + 16) * lr.U  # sums over rows, whatever their order, with the totals of several units
    for lo, hi, k in c.pieces:
        A, B, s = p["A"][k].double(), p["B"][k].double(), lr.scale_of(p, k)
        x, dy, e = X[lo:hi], d[lo:hi], ed[lo:hi]
        v, dv = s * (x @ A), s * (dy @ B.t())
        ev = (c.h_in + 8) * lr.U * s * (x.abs() @ A.abs())
        edv = s * (e @ B.abs().t()) + (c.h_out + 8) * lr.U * s * (dy.abs() @ B.abs().t())
        sv = ev + h * h * v.abs() + lr.lo_floor(c.dtype, v, ev)
        sdv = edv + h * h * dv.abs() + lr.lo_floor(c.dtype, dv, edv)
        dA[k] += x.t() @ dv
        eA[k] += x.abs().t() @ sdv + n * (x.abs().t() @ dv.abs())
        dB[k] += v.t() @ dy
        eB[k] += sv.t() @ dy.abs() + v.abs().t() @ e + n * (v.abs().t() @ dy.abs())
    return list(zip(dA, eA)), list(zip(dB, eB))


def check(got, ref, bound, dtype, what):
    """lr.check where the exact value stays inside fp16's range.  Rounding to nearest turns values from 65520 on (half a
    step past the largest finite 65504) into infinities: there the result is that infinity, and either within the bound of it."""
    over, under = ref.abs() - bound >= 65520, ref.abs() + bound < 65520
    infinite = torch.where(ref > 0, float("inf"), float("-inf"))
    assert torch.equal(got.double()[over], infinite[over]), f"{what}: values beyond the format"
    edge = ~over & ~under & (got.double() == infinite)
    lr.check(torch.where(over | edge, 0.0, got.double()), torch.where(over | edge, 0.0, ref), bound, dtype, what)


def spread(c, side, ratio, where):
    """Rows of dY (side "dA") or X ("dB") larger by 2^ratio, half of it on either side of 1: the first ones, the last
    ones or every third.  In the other operand the large rows have zeros in the even columns: in those columns of the
    gradient the small rows are all there is."""
    large = {"first": range(0, c.n // 3), "last": range(c.n - c.n // 3, c.n), "every_third": range(0, c.n, 3)}[where]
    big = torch.zeros(c.n, dtype=torch.bool, device="cuda")
    big[list(large)] = True
    step = torch.where(big, 2.0 ** (ratio // 2), 2.0 ** -(ratio - ratio // 2))[:, None].half()
    scaled, other = (c.dY, c.X) if side == "dA" else (c.X, c.dY)
    scaled.mul_(step)
    other[:, ::2] *= (~big[:, None]).half()


@pytest.mark.parametrize("side", ["dA", "dB"])
@pytest.mark.parametrize("where", ["first", "last", "every_third"])
@pytest.mark.parametrize("ratio", [12, 16, 20])
@pytest.mark.parametrize("n,rank", [(70, 64), (333, 16), (97, 8), (130, 32)])
def test_lora_gradients_of_rows_far_apart(n, rank, ratio, where, side):
    c = lr.Layer(101 + ratio, "f16", n, 136, 264, rank, 3, "mixed", 1, None, True)
    spread(c, side, ratio, where)
    _, grads = run_dense_back(c, "f16", train_w=False)
    d = c.dY.double()
    for name, got, refs in zip(("dA", "dB"), grads[0][1:3], lora_gradients(c, c.proj[0], d, torch.zeros_like(d))):
        for k in range(c.P):
            check(got[k], *refs[k], c.dtype, f"{name}[{k}]")


def test_rows_of_zeros_and_of_infinities_among_others():
    """Rows of zeros have no unit and disturb nobody; an infinity stays in the columns and the LoRA that it reaches."""
    c = lr.Layer(7, "f16", 120, 136, 72, 16, 2, "none", 1, None, False)
    c.seg, c.ids = [0, 70, 120], [0, 1]
    spread(c, "dA", 16, "every_third")
    c.X[5:20] = 0
    c.dY[11:33] = 0
    c.X[64:70] = 0
    d = c.dY.double()
    want = lora_gradients(c, c.proj[0], d, torch.zeros_like(d))
    _, grads = run_dense_back(c, "f16", train_w=False)
    for got, refs in zip(grads[0][1:3], want):
        for k in range(2):
            lr.check(got[k], *refs[k], c.dtype, f"LoRA {k}")
    c.X[40, 3] = float("inf")       # V of row 40 is infinite; X's column 3 as well
    _, broken = run_dense_back(c, "f16", train_w=False)
    assert torch.equal(broken[0][1][1], grads[0][1][1]) and torch.equal(broken[0][2][1], grads[0][2][1])
    others = [i for i in range(c.h_in) if i != 3]
    assert torch.equal(broken[0][1][0][others], grads[0][1][0][others])
    assert not torch.isfinite(broken[0][1][0][3]).any()


def gate_backward(c, kind):
    """dG, dU in 64 bits from the stored G, U and dH, the bounds of the values that the products read, and the unit of
    the largest row.  A row of both is kept in the unit 2^(8 b) that puts its largest |dH| max(1.13 |U|, |G|) into
    [2^7, 2^15): rounded once there (h, or h^2 as two halves), or by half of fp16's smallest denormal, 2^-25 units."""
    h = lr.half_step(c.dtype)
    g, u, dh = c.proj[0]["G"].double(), c.proj[1]["G"].double(), c.dY.double()
    a, slope = lr.act(kind, g)
    dg, du = dh * u * slope, dh * a
    if c.n <= 128 and c.n * c.h_out <= 2 ** 18:
        h = h * h
    eg = 2.0 ** -20 * (dh * u).abs() * 1.13 * (1 + g.abs())
    eu = 2.0 ** -20 * (dh * g).abs()
    big = (dh.abs() * torch.maximum(1.13 * u.abs(), g.abs())).amax(1) * (1 + 2.0 ** -20)
    power = torch.div(torch.frexp(big).exponent - 1 - 7, 8, rounding_mode="floor").clamp(-15, 15)
    unit = torch.where(big > 0, 2.0 ** (8.0 * power.double()), 0.0)[:, None]
    return (dg, eg + h * dg.abs() + 2.0 ** -25 * unit), (du, eu + h * du.abs() + 2.0 ** -25 * unit), float(unit.max())


MAGNITUDES = {"beyond": [(10, 8)], "small": [(-12, 0)], "both": [(10, 8), (-12, 0), (-4, -6)]}  # of dH and U, as 2^m
SIZES = {  # n, h_in, h_out: waves or workgroups per row, few rows as halves, rows longer than what a workgroup holds
    "few": (77, 136, 264), "one": (1, 72, 520), "rows": (300, 136, 264), "wide_few": (20, 136, 2056),
    "waves": (1100, 72, 1048), "wide": (600, 136, 2056), "wide4": (600, 72, 5000), "wide6": (520, 72, 12280),
    "wider": (520, 72, 12296), "widest": (515, 16, 26000), "middle": (150, 72, 4200), "widest_few": (20, 72, 16648),
}


@pytest.mark.parametrize("act", [sg.SGMV_ACT_SILU, sg.SGMV_ACT_GELU_TANH])
@pytest.mark.parametrize("magnitude", sorted(MAGNITUDES))
@pytest.mark.parametrize("size", sorted(SIZES))
def test_gated_gradients_beyond_fp16_and_far_below(size, magnitude, act):
    """dG and dU past 65504, or so small that fp16 would cut them, or both in one batch: gradients that fit come out right."""
    n, h_in, h_out = SIZES[size]
    c = lr.Layer(131, "f16", n, h_in, h_out, 16, 3, "mixed", 2, None, True)
    steps = MAGNITUDES[magnitude]
    power = torch.tensor([steps[i % len(steps)] for i in range(n)], device="cuda").double()
    c.dY.copy_((c.dY.double() * 2.0 ** power[:, :1]).half())
    c.proj[1]["G"].copy_((c.proj[1]["G"].double() * 2.0 ** power[:, 1:]).half())
    if magnitude != "small":        # outputs of the large rows stay in the format
        c.X.mul_(2.0 ** -8)
        for p in c.proj:
            p["W"].mul_(2.0 ** -8)
            for k in range(c.P):
                p["B"][k].mul_(2.0 ** -8)
    if n > 4:
        c.dY[n // 2] = 0            # a row of zeros
    dX, grads = run_gated_back(c, "f16", act)
    dg, du, top = gate_backward(c, act)
    ref = bound = 0
    for i, (p, d) in enumerate(zip(c.proj, (dg, du))):
        (x, ex), _, _, (w, ew) = lr.backward(c, p, *d)
        ref, bound = ref + x, bound + ex
        halves = 2 if n <= 128 and n * h_out <= 2 ** 18 else 1
        ew = ew + halves * 2.0 ** -25 * top * c.X.double().abs().sum(0)[:, None]     # rows brought to the largest unit
        check(grads[i][0], w, ew, c.dtype, f"dW[{i}]")
        for name, got, refs in zip(("dA", "dB"), grads[i][1:3], lora_gradients(c, p, *d)):
            for k in range(c.P):
                check(got[k], *refs[k], c.dtype, f"{name}[{i}][{k}]")
    check(dX, ref, bound, c.dtype, "dX")


def test_an_infinite_row_of_the_gated_block_stays_its_own():
    """An infinite dH reaches its row of dX, its LoRA and dW; other rows and LoRAs keep their values bit for bit."""
    c = lr.Layer(9, "f16", 200, 136, 264, 16, 2, "none", 2, None, False)
    c.seg, c.ids = [0, 90, 200], [0, 1]
    dX, grads = run_gated_back(c, "f16", 0)
    c.dY[30, 5] = float("inf")
    broken, other = run_gated_back(c, "f16", 0)
    rows = [i for i in range(200) if i != 30]
    assert torch.equal(broken[rows], dX[rows]) and not torch.isfinite(broken[30]).any()
    for i in range(2):
        assert torch.equal(other[i][1][1], grads[i][1][1]) and torch.equal(other[i][2][1], grads[i][2][1])
        columns = [j for j in range(264) if j != 5]
        assert torch.equal(other[i][0][:, columns], grads[i][0][:, columns])
