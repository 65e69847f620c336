"""GPU parity of the layer norm and its gradients against 64 bits, element by element, within derived bounds.

Bounds, with u = 2^-24 (half a step of fp32) and h half a step of the 16-bit format: a sum over the row takes at most D
additions one after another for any of its terms (8 values an eight, up to 4 eights a lane, 6 steps over a wave, 16 waves: 54; wide rows,
1024 lanes: 8 for every 8192 columns and 22), so it is off by (D + 2) u of its terms' absolute sum.  Sums over rows: D rows one after
another per workgroup and 64 to join (wide rows: any split, so n).  Everything else is a rounding or two of the terms named below."""
import pytest
import torch

import segmented_gather_matvec_amd as sg

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def depth(w):
    return 54 + w // 1024 + 24


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134


def check(got, ref, bound, what):
    if got.dtype != torch.float32:
        bound = bound + torch.finfo(got.dtype).eps / 2 * (ref.abs() + bound) + tiny(got.dtype)
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite"
    err = (got.double() - ref).abs()
    bad = err > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, worst err / bound {float((err / bound).max()):.3g}"


class Case:
    def __init__(self, seed, dtype, n, w, scale=1.0, shift=0.0, gamma=True, beta=True, eps=1e-5):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.n, self.w, self.eps = DT[dtype], n, w, eps
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        big = 1 + 15 * (torch.rand(w, generator=g) < 0.05)
        to = lambda t: t.to(self.dtype).cuda()  # noqa: E731
        self.X = to((r(n, w) * big + 0.5 * r(n, 1)) * scale + shift)
        self.gamma, self.beta = to(1 + 0.3 * r(w)) if gamma else None, to(r(w)) if beta else None
        self.dY, self.beyond = to(r(n, w)), to(r(n, w))

    def nan(self, *shape, dtype=None):
        return torch.full(shape, float("nan"), dtype=dtype or self.dtype, device="cuda")

    def forward(self):
        Y, mean, rstd = self.nan(self.n, self.w), self.nan(self.n, dtype=torch.float32), self.nan(self.n, dtype=torch.float32)
        sg.sgmv_layer_norm_apply(self.X, self.gamma, self.beta, Y, self.eps, mean=mean, rstd=rstd)
        return Y, mean, rstd

    def backward(self, mean, rstd, beyond=True, accumulate=False, fill=float("nan")):
        ws = sg.new_layer_norm_workspace(self.n, self.w)
        ws.fill_(0xFF)
        dX = self.nan(self.n, self.w)
        dg, db = (torch.full((self.w,), fill, dtype=self.dtype, device="cuda") for _ in range(2))
        sg.sgmv_layer_norm_backward(self.X, self.gamma, mean, rstd, self.dY, ws, dX=dX,
                                    beyond=self.beyond if beyond else None, dgamma=dg, dbeta=db, accumulate=accumulate)
        return dX, dg, db

    # 64 bits: values and the bounds of what is not rounded to 16 bits yet
    def moments(self):
        x = self.X.double()
        mean = x.mean(1)
        em = (depth(self.w) + 2) * u * x.abs().mean(1)
        d = x - mean[:, None]
        var = (d * d).mean(1)
        ev = em * em + (depth(self.w) + 8) * u * (var + em * em)
        rstd = (var + self.eps) ** -0.5
        er = 0.5 * ev / (var + self.eps) / (1 - ev / (var + self.eps)).clamp(min=0.1) + 6 * u       # relative
        return mean, em, rstd, er

    def ref_forward(self):
        mean, em, rstd, er = self.moments()
        g = self.gamma.double() if self.gamma is not None else torch.ones(self.w, dtype=torch.float64, device="cuda")
        b = self.beta.double() if self.beta is not None else torch.zeros(self.w, dtype=torch.float64, device="cuda")
        d = self.X.double() - mean[:, None]
        y = d * rstd[:, None] * g + b
        ey = g.abs() * rstd[:, None] * (em[:, None] + (d.abs() + em[:, None]) * (er[:, None] + 5 * u)) + 2 * u * (b.abs() + y.abs())
        return (y, ey), (mean, em + 2 * u * mean.abs()), (rstd, rstd * er)

    def ref_backward(self, mean, rstd, beyond=True):
        x, dy, r, D = self.X.double(), self.dY.double(), rstd.double()[:, None], depth(self.w)
        g = self.gamma.double() if self.gamma is not None else torch.ones(self.w, dtype=torch.float64, device="cuda")
        xh, q = (x - mean.double()[:, None]) * r, dy * g
        m0, m1 = q.mean(1, keepdim=True), (q * xh).mean(1, keepdim=True)
        e0, e1 = (D + 4) * u * q.abs().mean(1, keepdim=True), (D + 8) * u * (q * xh).abs().mean(1, keepdim=True)
        dx = r * (q - m0 - xh * m1)
        ex = r * (e0 + xh.abs() * e1 + 6 * u * (q.abs() + m0.abs() + (xh * m1).abs()))
        if beyond:
            dx = dx + self.beyond.double()
            ex = ex + 2 * u * (dx.abs() + self.beyond.double().abs())
        R = (self.n if self.w > 12288 else self.n // 512) + 64 + 16
        return ((dx, ex), ((dy * xh).sum(0), (R + 4) * u * (dy * xh).abs().sum(0)), (dy.sum(0), R * u * dy.abs().sum(0)))


# Every variant of rows held in registers, either side of its widest row, and rows that are read again; one row to many.
SIZES = [(1, 8), (3, 64), (5, 512), (9, 520), (64, 1024), (17, 1032), (33, 2048), (7, 2056), (300, 4096), (130, 4104), (21, 6152),
         (40, 8192), (5, 8200), (3, 12288), (9, 12296), (5, 16384), (4, 16392), (3, 24576), (2, 24584), (2, 1 << 17), (1, 1 << 20),
         (2500, 264), (1100, 4096), (700, 8200), (70, 14008)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,w", SIZES)
def test_norm_and_gradients(n, w, dtype):
    c = Case(n * 31 + w, dtype, n, w)
    got = c.forward()
    for g, (ref, bound), what in zip(got, c.ref_forward(), ("Y", "mean", "rstd")):
        check(g, ref, bound, what)
    dX, dg, db = c.backward(*got[1:])
    for g, (ref, bound), what in zip((dX, dg, db), c.ref_backward(*got[1:]), ("dX", "dgamma", "dbeta")):
        check(g, ref, bound, what)


@pytest.mark.parametrize("gamma,beta", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("n,w", [(6, 136), (11, 4104), (3, 30008)])
def test_without_parameters(n, w, gamma, beta):
    c = Case(5, "bf16", n, w, gamma=gamma, beta=beta)
    Y, mean, rstd = c.forward()
    check(Y, *c.ref_forward()[0], "Y")
    plain = c.nan(n, w)
    sg.sgmv_layer_norm_apply(c.X, c.gamma, c.beta, plain, c.eps)         # moments not wanted
    assert torch.equal(plain, Y)
    dX, dg, db = c.backward(mean, rstd, beyond=False)
    for g, (ref, bound), what in zip((dX, dg, db), c.ref_backward(mean, rstd, beyond=False), ("dX", "dgamma", "dbeta")):
        check(g, ref, bound, what)


# Rows of four eights a lane, several to a workgroup, whose gamma stays in LDS; gradients over their own inputs.
@pytest.mark.parametrize("gamma", [False, True])
@pytest.mark.parametrize("n,w,dtype", [(600, 12296, "bf16"), (520, 14344, "f16"), (300, 16384, "bf16")])
def test_wide_rows_one_after_another(n, w, dtype, gamma):
    c = Case(n + w, dtype, n, w, gamma=gamma)
    _, mean, rstd = c.forward()
    dX, dg, db = c.backward(mean, rstd)
    for g, (ref, bound), what in zip((dX, dg, db), c.ref_backward(mean, rstd), ("dX", "dgamma", "dbeta")):
        check(g, ref, bound, what)
    ws = sg.new_layer_norm_workspace(n, w)
    for into in ("dY", "beyond"):
        t = getattr(c, into).clone()
        sg.sgmv_layer_norm_backward(c.X, c.gamma, mean, rstd, t if into == "dY" else c.dY, ws, dX=t,
                                    beyond=t if into == "beyond" else c.beyond)
        assert torch.equal(t, dX)


@pytest.mark.parametrize("w", [520, 4096, 40000])
@pytest.mark.parametrize("scale,shift", [(2.0 ** -9, 0.0), (1.0, 300.0), (2.0 ** -6, -40.0), (500.0, 0.0), (2.0 ** -20, 0.0)])
def test_small_large_and_shifted_rows(w, scale, shift):
    """A mean far from 0 must not cost the variance its bits; tiny rows meet eps."""
    c = Case(17, "f16" if shift else "bf16", 6, w, scale, shift)
    got = c.forward()
    for g, (ref, bound), what in zip(got, c.ref_forward(), ("Y", "mean", "rstd")):
        check(g, ref, bound, what)
    for g, (ref, bound), what in zip(c.backward(*got[1:]), c.ref_backward(*got[1:]), ("dX", "dgamma", "dbeta")):
        check(g, ref, bound, what)


@pytest.mark.parametrize("w", [256, 5120, 26000])
def test_constant_rows_and_rows_that_are_not_finite(w):
    """A constant row is beta; a row with an infinity or NaN spoils itself (and the parameters' gradients) only."""
    c = Case(23, "f16", 9, w)
    clean = c.forward()
    clean_dX = c.backward(*clean[1:])[0]
    c.X[3] = 1.5
    c.X[5, w // 2] = float("inf")
    c.X[7, w - 1] = float("nan")
    Y, mean, rstd = c.forward()
    assert torch.equal(Y[3], c.beta) and float(mean[3]) == 1.5
    assert Y[5].isnan().any() and Y[7].isnan().all()
    keep = [0, 1, 2, 4, 6, 8]
    for a, b in zip((Y, mean, rstd), clean):
        assert torch.equal(a[keep], b[keep])
    dX, dg, db = c.backward(mean, rstd)
    assert torch.equal(dX[keep], clean_dX[keep]) and torch.isfinite(dX[3].float()).all()
    assert dg.isnan().any() and torch.isfinite(db.float()).all()


@pytest.mark.parametrize("w", [136, 4096, 20000])
def test_parts_in_place_and_accumulation(w):
    c = Case(29, "bf16", 37, w)
    Y, mean, rstd = c.forward()
    X = c.X.clone()
    sg.sgmv_layer_norm_apply(X, c.gamma, c.beta, X, c.eps)
    assert torch.equal(X, Y)
    dX, dg, db = c.backward(mean, rstd)
    ws = sg.new_layer_norm_workspace(c.n, w)

    def run(**kw):
        ws.fill_(0xFF)
        sg.sgmv_layer_norm_backward(c.X, c.gamma, mean, rstd, kw.pop("dY", c.dY), ws, **{"beyond": c.beyond, **kw})

    for into in ("dY", "beyond"):
        t = (c.dY if into == "dY" else c.beyond).clone()
        run(dX=t, **{into: t})
        assert torch.equal(t, dX)
    for name, want in (("dX", dX), ("dgamma", dg), ("dbeta", db)):
        t = torch.full_like(want, float("nan"))
        run(**{name: t})
        assert torch.equal(t, want)
    _, ag, ab = c.backward(mean, rstd, accumulate=True, fill=3.0)
    _, (rg, eg), (rb, eb) = c.ref_backward(mean, rstd)
    check(ag, rg + 3, eg + 2 * u * (rg.abs() + 3), "dgamma")
    check(ab, rb + 3, eb + 2 * u * (rb.abs() + 3), "dbeta")


@pytest.mark.parametrize("accumulate", [False, True])
def test_no_rows(accumulate):
    c = Case(1, "f16", 0, 264)
    dX, dg, db = c.backward(torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), accumulate=accumulate, fill=2.0)
    assert (dg == (2.0 if accumulate else 0.0)).all() and (db == (2.0 if accumulate else 0.0)).all()
    assert c.forward()[0].shape == (0, 264)


@pytest.mark.parametrize("w", [72, 1000, 13000])
def test_gradient_against_differences(w):
    """Directional derivatives of the 64-bit norm by central differences, eps 1e-4 (their own error, third derivatives
    times 1e-8, is far below the bound of 16-bit gradients along a random direction)."""
    c = Case(41, "f16", 5, w)
    _, mean, rstd = c.forward()
    dX, dg, db = c.backward(mean, rstd, beyond=False)
    refs = c.ref_backward(mean, rstd, beyond=False)
    # (The stored moments are fp32: off by their bounds, which move the formula's dX by as much again.)
    _, em, _, er = c.moments()
    gen = torch.Generator(device="cuda").manual_seed(3)

    def loss(x, g, b):
        d = x - x.mean(1, keepdim=True)
        return float(((d * ((d * d).mean(1, keepdim=True) + c.eps) ** -0.5 * g + b) * c.dY.double()).sum())

    base = (c.X.double(), c.gamma.double(), c.beta.double())
    for i, got in enumerate((dX, dg, db)):
        v = torch.randn(base[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        plus, minus = ([t + s * 1e-4 * v if j == i else t for j, t in enumerate(base)] for s in (1, -1))
        diff = (loss(*plus) - loss(*minus)) / 2e-4
        ref, bound = refs[i]
        moved = 8 * ((em * rstd.double() + er).max()) * (ref.abs() + ref.abs().mean())
        bound = ((bound + moved + torch.finfo(c.dtype).eps / 2 * (ref.abs() + bound)) * v.abs()).sum()
        assert abs(float((got.double() * v).sum()) - diff) <= float(bound) + 1e-6 * abs(diff)


@pytest.mark.parametrize("n,w", [(3, 520), (600, 4096), (40, 20000)])
def test_every_replay_writes_every_output(n, w):
    """Forward and backward captured once; every output and the workspace overwritten before each replay, eager calls between."""
    c = Case(51, "bf16", n, w)
    want = c.forward()
    want = want + c.backward(*want[1:])
    out = [torch.empty_like(t) for t in want]
    ws = sg.new_layer_norm_workspace(n, w)

    def step():
        sg.sgmv_layer_norm_apply(c.X, c.gamma, c.beta, out[0], c.eps, mean=out[1], rstd=out[2])
        sg.sgmv_layer_norm_backward(c.X, c.gamma, out[1], out[2], c.dY, ws, dX=out[3], beyond=c.beyond, dgamma=out[4], dbeta=out[5])

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
        ws.fill_(0xFF)
        graph.replay()
        c.forward()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once():
    a, b = Case(61, "bf16", 900, 4096), Case(62, "f16", 50, 1000)
    wants = []
    for c in (a, b):
        f = c.forward()
        wants.append(f + c.backward(*f[1:]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                f = c.forward()
                got.append(f + c.backward(*f[1:]))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(got, wants) for x, y in zip(g, w))
