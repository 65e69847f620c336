"""GPU tests of rows sorted by LoRA and back: the order, its inverse and the segments against a stable sort on the host, exactly;
dispatched rows exactly; combined rows and gradients against 64 bits, within h (half a step of the format) of an output's one
rounding and, of fp32 sums, (terms one after another) x 2^-24 of the terms' absolute sum."""
import numpy as np
import pytest
import torch

import segmented_gather_matvec_amd as sg

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
I32 = torch.int32


def route(ids, P):
    n, k = ids.shape
    m = n * k
    perm, slots, seg, idx = (torch.full((s,), -7, dtype=I32, device="cuda") for s in (m, m, P + 1, P))
    ws = sg.new_route_workspace(n, k, P)
    if ws.numel():
        ws.fill_(0xFF)
    sg.sgmv_route_rows(ids, P, perm, slots, seg, idx, ws)
    return perm, slots, seg, idx


def expected(ids, P):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < P), flat, P)
    perm = np.argsort(key, kind="stable")
    slots = np.empty_like(perm)
    slots[perm] = np.arange(perm.size)
    return perm, slots, np.searchsorted(key[perm], np.arange(P + 1), side="left")


def choices(kind, n, k, P, seed):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        ids = rng.integers(0, P, size=(n, k))
    elif kind == "one":
        ids = np.full((n, k), P - 1)
    elif kind == "none":
        ids = np.full((n, k), -1)
    elif kind == "skewed":
        ids = np.minimum(rng.zipf(1.4, size=(n, k)) - 1, P - 1)
    else:       # some without a LoRA, in every way that says so
        ids = rng.integers(0, P, size=(n, k))
        odd = rng.choice(np.array([-1, P, P + 1, -2 ** 31, 2 ** 31 - 1]), size=(n, k))
        ids = np.where(rng.random((n, k)) < 0.3, odd, ids)
    return torch.from_numpy(ids.astype(np.int32)).cuda()


# One workgroup and several, either side of a tile's edge, few and many LoRAs (fewer waves a workgroup), top_k up to the most.
ROUTES = [(1, 1, 1), (1, 2, 3), (7, 1, 8192), (32, 2, 32), (63, 1, 5), (64, 1, 5), (65, 3, 64), (1023, 1, 63), (1024, 1, 2), (1025, 1, 64),
          (2048, 1, 16), (2049, 1, 16), (4096, 2, 8), (5000, 3, 511), (777, 64, 40), (3001, 8, 2400), (20000, 1, 8192), (9000, 8, 3),
          (150000, 2, 100), (1 << 20, 1, 1000)]


@pytest.mark.parametrize("kind", ["uniform", "one", "none", "skewed", "some_without"])
@pytest.mark.parametrize("n,k,P", ROUTES)
def test_order_inverse_and_segments(n, k, P, kind):
    ids = choices(kind, n, k, P, n + P)
    perm, slots, seg, idx = route(ids, P)
    wp, ws, wb = expected(ids, P)
    assert np.array_equal(perm.cpu().numpy(), wp)
    assert np.array_equal(slots.cpu().numpy(), ws)
    assert np.array_equal(seg.cpu().numpy(), wb)
    assert np.array_equal(idx.cpu().numpy(), np.arange(P))


def test_matches_the_host_builder():
    """One LoRA a row: the host builder's perm, and its segments where they are not empty."""
    req = np.random.default_rng(3).integers(0, 40, size=500)
    perm, seg, lidx, _ = sg.sgmv_build_segments(req, 60)
    got = route(torch.from_numpy(req.astype(np.int32)).cuda()[:, None], 60)
    assert np.array_equal(got[0].cpu().numpy(), perm)
    bounds = got[2].cpu().numpy()
    full = np.flatnonzero(np.diff(bounds))
    assert np.array_equal(full, lidx) and np.array_equal(np.append(bounds[:-1][full], 500), seg)


def test_outputs_are_optional_and_no_rows_give_empty_segments():
    ids = choices("some_without", 3000, 2, 50, 9)
    want = route(ids, 50)
    for i in range(4):
        out = [None] * 4
        out[i] = torch.full_like(want[i], -7)
        sg.sgmv_route_rows(ids, 50, *out, sg.new_route_workspace(3000, 2, 50))
        assert torch.equal(out[i], want[i])
    _, _, seg, idx = route(torch.empty(0, 2, dtype=I32, device="cuda"), 50)
    assert (seg == 0).all() and torch.equal(idx, torch.arange(50, dtype=I32, device="cuda"))


@pytest.mark.parametrize("n,P", [(900, 40), (7000, 40)])
def test_an_order_over_its_own_ids_stays_inside(n, P):
    """perm written over ids, which the header forbids: the values are anything, the neighbours are not touched."""
    buffer = torch.full((n + 128,), 12345, dtype=I32, device="cuda")
    ids = buffer[64:64 + n]
    ids.copy_(choices("uniform", n, 1, P, 3)[:, 0])
    slots = torch.full((n + 128,), 12345, dtype=I32, device="cuda")
    sg.sgmv_route_rows(ids, P, ids, slots[64:64 + n], None, None, sg.new_route_workspace(n, 1, P))
    for t in (buffer, slots):
        assert (t[:64] == 12345).all() and (t[-64:] == 12345).all()


class Rows:
    def __init__(self, seed, dtype, n, k, w, P=5):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.n, self.k, self.w, self.m = DT[dtype], n, k, w, n * k
        r = lambda *s: torch.randn(*s, generator=g).to(self.dtype).cuda()  # noqa: E731
        self.X, self.R, self.dY, self.Ys, self.dXs = r(n, w), r(n, w), r(n, w), r(self.m, w), r(self.m, w)
        self.weights = torch.rand(n, k, generator=g).cuda()
        self.weights[torch.rand(n, k, generator=g) < 0.1] = 0
        self.slots = route(choices("some_without", n, k, P, seed), P)[1]
        self.at = self.slots.long().reshape(n, k)

    def nan(self, *shape, dtype=None):
        return torch.full(shape, float("nan"), dtype=dtype or self.dtype, device="cuda")


def check(got, ref, bound, what):
    if got.dtype != torch.float32:
        bound = bound + torch.finfo(got.dtype).eps / 2 * (ref.abs() + bound) + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -134)
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite"
    err = (got.double() - ref).abs()
    bad = err > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, worst err / bound {float((err / bound).max()):.3g}"


def run_combine(c, Ys, weights=None, residual=None):
    Y = c.nan(c.n, c.w)
    sg.sgmv_combine_rows(Ys, c.slots, Y, weights=weights, residual=residual)
    return Y


def ref_combine(c, Ys, weights=None, residual=None):
    w = weights.double()[:, :, None] if weights is not None else 1.0
    terms = w * Ys.double()[c.at]
    y, mag = terms.sum(1), terms.abs().sum(1)
    if residual is not None:
        y, mag = y + residual.double(), mag + residual.double().abs()
    return y, (c.k + 1) * u * mag


SIZES = [(1, 1, 8), (1, 2, 4096), (2, 3, 56), (5, 2, 64), (33, 1, 72), (9, 4, 136), (40, 2, 264), (65, 5, 520), (130, 8, 1032),
         (257, 2, 4104), (3, 64, 512), (2100, 1, 136), (1500, 2, 2056), (2, 2, 40008), (1, 3, 1 << 20)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,k,w", SIZES)
def test_rows_out_and_back(n, k, w, dtype):
    c = Rows(n + k + w, dtype, n, k, w)
    Xs = c.nan(c.m, w)
    sg.sgmv_dispatch_rows(c.X, c.slots, Xs)
    assert torch.equal(Xs[c.at.reshape(-1)], c.X.repeat_interleave(k, 0))
    for weights in (None, c.weights):
        for residual in (None, c.R):
            check(run_combine(c, c.Ys, weights, residual), *ref_combine(c, c.Ys, weights, residual), "Y")
        dYs, dw = c.nan(c.m, w), c.nan(n, k, dtype=torch.float32)
        sg.sgmv_combine_rows_backward(c.dY, c.Ys, c.slots, weights=weights, dYs=dYs, dweights=dw)
        dy, ww = c.dY.double(), weights.double() if weights is not None else torch.ones(n, k, dtype=torch.float64, device="cuda")
        want = (ww[:, :, None] * dy[:, None, :]).reshape(c.m, w)
        check(dYs[c.at.reshape(-1)], want, u * want.abs(), "dYs")
        products = dy[:, None, :] * c.Ys.double()[c.at]
        check(dw, products.sum(2), (w // 64 + 32) * u * products.abs().sum(2), "dweights")


def test_gradient_of_dispatch_is_combine():
    """<dXs, dispatch(X)> = <combine(dXs), X> up to the rounding of combine's output (h of it, and u a term)."""
    c = Rows(3, "bf16", 90, 3, 136)
    dX = run_combine(c, c.dXs)
    Xs = c.nan(c.m, c.w)
    sg.sgmv_dispatch_rows(c.X, c.slots, Xs)
    ref, bound = ref_combine(c, c.dXs)
    off = ((bound + 2.0 ** -8 * (ref.abs() + bound)) * c.X.double().abs()).sum()
    assert abs(float((c.dXs.double() * Xs.double()).sum() - (dX.double() * c.X.double()).sum())) <= float(off)


def test_gradients_against_differences():
    """Combine is linear in Ys and in the weights: a difference quotient of the 64-bit sum is the derivative but for rounding."""
    c = Rows(4, "f16", 20, 4, 200)
    dYs, dw = c.nan(c.m, c.w), c.nan(20, 4, dtype=torch.float32)
    sg.sgmv_combine_rows_backward(c.dY, c.Ys, c.slots, weights=c.weights, dYs=dYs, dweights=dw)
    gen = torch.Generator(device="cuda").manual_seed(1)
    loss = lambda ys, w: float(((w[:, :, None] * ys[c.at]).sum(1) * c.dY.double()).sum())  # noqa: E731
    ys, w = c.Ys.double(), c.weights.double()
    v = torch.randn(ys.shape, generator=gen, device="cuda", dtype=torch.float64)
    diff = (loss(ys + v, w) - loss(ys - v, w)) / 2
    assert abs(float((dYs.double() * v).sum()) - diff) <= float((2.0 ** -11 * 1.01 * dYs.double() * v).abs().sum()) + 1e-9
    v = torch.randn(w.shape, generator=gen, device="cuda", dtype=torch.float64)
    diff = (loss(ys, w + v) - loss(ys, w - v)) / 2
    size = (c.dY.double()[:, None, :] * ys[c.at]).abs().sum(2)
    assert abs(float((dw.double() * v).sum()) - diff) <= float((40 * u * size * v.abs()).sum()) + 1e-9


def test_a_weight_of_zero_hides_its_row():
    c = Rows(5, "f16", 30, 2, 264)
    c.weights[4, 1] = c.weights[9, 0] = 0
    Y = run_combine(c, c.Ys, c.weights, c.R)
    bad = c.Ys.clone()
    bad[c.at[4, 1]], bad[c.at[9, 0]] = float("nan"), float("inf")
    assert torch.equal(run_combine(c, bad, c.weights, c.R), Y)
    dY = c.dY.clone()
    dY[4] = float("inf")
    dYs = c.nan(c.m, c.w)
    sg.sgmv_combine_rows_backward(dY, None, c.slots, weights=c.weights, dYs=dYs)
    assert (dYs[c.at[4, 1]] == 0).all()


def test_in_place_residual_and_parts():
    c = Rows(6, "bf16", 70, 2, 1032)
    Y = run_combine(c, c.Ys, c.weights, c.R)
    R = c.R.clone()
    sg.sgmv_combine_rows(c.Ys, c.slots, R, weights=c.weights, residual=R)
    assert torch.equal(R, Y)
    dYs, dw = c.nan(c.m, c.w), c.nan(70, 2, dtype=torch.float32)
    sg.sgmv_combine_rows_backward(c.dY, c.Ys, c.slots, weights=c.weights, dYs=dYs, dweights=dw)
    a, b = torch.full_like(dYs, 7.0), torch.full_like(dw, 7.0)
    sg.sgmv_combine_rows_backward(c.dY, None, c.slots, weights=c.weights, dYs=a)
    sg.sgmv_combine_rows_backward(c.dY, c.Ys, c.slots, weights=c.weights, dweights=b)
    assert torch.equal(a, dYs) and torch.equal(b, dw)


def test_places_outside_are_passed_over():
    """slots that no sort made: entries outside the rows fill and add nothing, their neighbours are right."""
    c = Rows(7, "f16", 12, 2, 136)
    c.slots[5], c.slots[11] = -1, c.m
    at = c.slots.long()
    Xs = torch.full((c.m + 2, c.w), 7.0, dtype=c.dtype, device="cuda")
    sg.sgmv_dispatch_rows(c.X, c.slots, Xs[1:-1])
    inside = (at >= 0) & (at < c.m)
    assert torch.equal(Xs[1:-1][at[inside]], c.X.repeat_interleave(2, 0)[inside])
    assert (Xs[0] == 7).all() and (Xs[-1] == 7).all() and int((Xs[1:-1] == 7).all(1).sum()) == 2
    w = torch.where(inside, 1.0, 0.0).reshape(12, 2).double()
    terms = w[:, :, None] * c.Ys.double()[at.clamp(0, c.m - 1).reshape(12, 2)]
    check(run_combine(c, c.Ys), terms.sum(1), 3 * u * terms.abs().sum(1), "Y")
    dYs, dw = torch.full((c.m + 2, c.w), 7.0, dtype=c.dtype, device="cuda"), c.nan(12, 2, dtype=torch.float32)
    sg.sgmv_combine_rows_backward(c.dY, c.Ys, c.slots, dYs=dYs[1:-1], dweights=dw)
    assert (dYs[0] == 7).all() and (dYs[-1] == 7).all() and int((dYs[1:-1] == 7).all(1).sum()) == 2
    assert (dw.reshape(-1)[~inside] == 0).all()


def test_every_replay_writes_every_output():
    c = Rows(8, "bf16", 2500, 2, 520, P=300)
    ids = choices("some_without", 2500, 2, 300, 77)

    def outputs():
        i32 = lambda s: torch.full((s,), -7, dtype=I32, device="cuda")  # noqa: E731
        return [i32(c.m), i32(c.m), i32(301), i32(300), c.nan(c.m, c.w), c.nan(c.n, c.w), c.nan(c.m, c.w),
                c.nan(c.n, 2, dtype=torch.float32)]

    ws = sg.new_route_workspace(2500, 2, 300)

    def step(o):
        sg.sgmv_route_rows(ids, 300, *o[:4], ws)
        sg.sgmv_dispatch_rows(c.X, o[1], o[4])
        sg.sgmv_combine_rows(o[4], o[1], o[5], weights=c.weights, residual=c.R)
        sg.sgmv_combine_rows_backward(c.dY, o[4], o[1], weights=c.weights, dYs=o[6], dweights=o[7])

    want, out = outputs(), outputs()
    step(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for _ in range(3):
        for t, f in zip(out, outputs()):
            t.copy_(f)
        ws.fill_(0xFF)
        graph.replay()
        route(ids, 300)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once():
    ids = [choices("skewed", 9000, 2, 64, 1), choices("uniform", 500, 1, 900, 2)]
    want = [route(i, P) for i, P in zip(ids, (64, 900))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for i, P, s in zip(ids, (64, 900), streams):
            with torch.cuda.stream(s):
                got.append(route(i, P))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
