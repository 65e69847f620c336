"""64-bit reference of the layer entry points (a shared projection with LoRA terms, the gated
feed-forward block, their gradients), segment by segment from the definition, with a bound
of what rounding may do to each output element.

Bounds, per element, with h = eps / 2 of the 16-bit format (half a step: 2^-8 bf16, 2^-11 fp16):
* an output's one rounding: h |value|;
* a sum of K products in fp32, in any order: (K + 8) 2^-23 sum |terms| (one unit in the last
  place per addition covers matrix cores that truncate);
* V = s x@A and dV = s dy@B^T enter matrix products as hi + lo halves: h^2 of each value, plus, in
  fp16, half of the smallest denormal (2^-25) where lo underflows, in units of the power 2^(16 b) that brings the row's largest
  value to [2^-4, 2^12).  The gradients of A_k and B_k sum rows in the LoRA's largest unit: bringing hi and lo there
  rounds each by another 2^-25 at most, 3 * 2^-25 < 2^-23 in all;
* dG, dU of the gated backward are rounded once: h of each; up to 128 rows and 2^18 values they are two halves: h^2;
* the activation in fp32: 2^-20 of the terms it is made of (exp and the divisions are good to a few
  units in the last place each).
Errors of intermediate values propagate through the absolute values of what multiplies them.
"""
import math

import numpy as np
import torch

U = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Layer:
    """Inputs of one case on the device, its segments on the host."""

    def __init__(self, seed, dtype, n, h_in, h_out, rank, P, layout, projections, ranks=None, scales=False,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        self.n, self.h_in, self.h_out, self.rank, self.P = n, h_in, h_out, rank, P

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g) * std).to(self.dtype).to(device)

        self.seg, self.ids = segments(layout, n, P, rng)
        self.X = normal(n, h_in)
        self.dY = normal(n, h_out)
        self.proj = []
        for _ in range(projections):
            rk = [rank] * P if ranks is None else [int(ranks[k % len(ranks)]) for k in range(P)]
            self.proj.append({
                "W": normal(h_in, h_out, std=h_in ** -0.5),
                "A": [normal(h_in, r, std=h_in ** -0.5) for r in rk],
                "B": [normal(r, h_out, std=max(1, r) ** -0.5) for r in rk],
                "ranks": rk if ranks is not None else None,
                "scales": (torch.rand(P, generator=g) + 0.5).to(device) if scales else None,
                "G": normal(n, h_out, std=1.4),
            })

    @property
    def pieces(self):
        return [(lo, hi, k) for lo, hi, k in zip(self.seg[:-1], self.seg[1:], self.ids) if hi > lo]


def segments(layout, n, P, rng):
    """(seg_indptr, lora_idx) as lists."""
    if layout == "none":
        return [0], []
    if layout == "one":
        return [0, n], [P - 1]
    if layout == "distinct":
        return list(range(n + 1)), [i % P for i in range(n)]
    if layout == "uncovered":           # the last third of the rows has no LoRA, the first segment is empty
        cut = max(1, 2 * n // 3)
        return [0, 0, cut // 2, cut, cut], [0, P - 1, 0, P // 2]
    if layout == "mixed":               # ragged, with empty segments and LoRAs used more than once
        S = max(2, min(n, 11))
        cuts = np.sort(rng.integers(0, n + 1, size=S - 1))
        return [0] + cuts.tolist() + [n], rng.integers(0, P, size=S).tolist()
    if layout == "many_empty":          # hundreds of empty segments around a few rows
        S = 700
        cuts = np.sort(rng.integers(0, n + 1, size=S - 1))
        return [0] + cuts.tolist() + [n], rng.integers(0, P, size=S).tolist()
    raise ValueError(layout)


def scale_of(p, k):
    return float(p["scales"][k]) if p["scales"] is not None else 1.0


def lo_floor(dtype, v, ev):
    """Per row of V (known up to ev): 2^-25 in the row's unit."""
    if dtype != torch.float16:
        return v.new_zeros(v.shape[0], 1)
    big = (v.abs() + ev).amax(1, keepdim=True) if v.shape[1] else v.new_zeros(v.shape[0], 1)
    exponent = torch.frexp(big).exponent - 1        # big in [2^exponent, 2^(exponent + 1)); fp32's range
    band = torch.div(exponent + 4, 16, rounding_mode="floor").clamp(-7, 7)
    return 2.0 ** -25 * torch.where(big > 0, 2.0 ** (16.0 * band.to(v.dtype)), 2.0 ** -112)


def project(c, p):
    """Y in 64 bits and the error bound of the unrounded fp32 sum."""
    h = half_step(c.dtype)
    X, W = c.X.double(), p["W"].double()
    y = X @ W
    err = (c.h_in + 8) * U * (X.abs() @ W.abs())
    for lo, hi, k in c.pieces:
        A, B, s = p["A"][k].double(), p["B"][k].double(), scale_of(p, k)
        x = X[lo:hi]
        v, va = s * (x @ A), s * (x.abs() @ A.abs())
        y[lo:hi] += v @ B
        ev = (c.h_in + 8) * U * va
        ev = ev + h * h * v.abs() + lo_floor(c.dtype, v, ev)
        err[lo:hi] += ev @ B.abs() + (c.rank + c.h_in + 16) * U * (v.abs() @ B.abs())
    return y, err


def act(kind, g):
    if kind == 0:
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * torch.sigmoid(-g))
    z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    s, t = torch.sigmoid(2 * z), torch.sigmoid(-2 * z)
    return g * s, s + 2 * math.sqrt(2 / math.pi) * g * s * t * (1 + 3 * 0.044715 * g * g)


def gate(c, kind):
    """H, G, U in 64 bits with the bounds of the stored values."""
    h = half_step(c.dtype)
    g, eg = project(c, c.proj[0])
    u, eu = project(c, c.proj[1])
    a, _ = act(kind, g)
    H = a * u
    # |act'| <= 1.13 for both activations
    eH = 1.13 * eg * (u.abs() + eu) + a.abs() * eu + 2.0 ** -20 * (g.abs() * u.abs())
    return [(H, eH + h * (H.abs() + eH)), (g, eg + h * (g.abs() + eg)), (u, eu + h * (u.abs() + eu))]


def backward(c, p, d, ed, train_w=True):
    """Gradients from the layer's output gradient d (64 bits) known up to ed, not rounded:
    dX, (dA_k), (dB_k), dW as (value, bound of the unrounded sum) pairs."""
    h = half_step(c.dtype)
    X, W = c.X.double(), p["W"].double()
    dX = d @ W.t()
    eX = ed @ W.abs().t() + (2 * c.h_out + 8) * U * (d.abs() @ W.abs().t())
    dA = [torch.zeros_like(a, dtype=torch.float64) for a in p["A"]]
    dB = [torch.zeros_like(b, dtype=torch.float64) for b in p["B"]]
    eA, eB = [torch.zeros_like(a) for a in dA], [torch.zeros_like(b) for b in dB]
    rows = [[] for _ in range(c.P)]
    for lo, hi, k in c.pieces:
        A, B, s = p["A"][k].double(), p["B"][k].double(), scale_of(p, k)
        x, dy, e = X[lo:hi], d[lo:hi], ed[lo:hi]
        v = s * (x @ A)
        ev = (c.h_in + 8) * U * s * (x.abs() @ A.abs())
        dv = s * (dy @ B.t())
        edv = s * (e @ B.abs().t()) + (c.h_out + 8) * U * s * (dy.abs() @ B.abs().t())
        sv, sdv = ev + h * h * v.abs(), edv + h * h * dv.abs()
        fv, fdv = lo_floor(c.dtype, v, ev), lo_floor(c.dtype, dv, edv)
        # What the sums over rows multiply, and the row's unit floor (the LoRA's largest comes below).
        rows[k].append((x.abs(), fdv, dy.abs(), fv))
        n = (2 * c.n + 16) * U  # sums over rows, LoRAs of several segments and splits among them
        dX[lo:hi] += dv @ A.t()
        eX[lo:hi] += (sdv + fdv) @ A.abs().t() + (c.rank + 16) * U * (dv.abs() @ A.abs().t())
        dA[k] += x.t() @ dv
        eA[k] += x.abs().t() @ sdv + n * (x.abs().t() @ dv.abs())
        dB[k] += v.t() @ dy
        eB[k] += sv.t() @ dy.abs() + v.abs().t() @ e + n * (v.abs().t() @ dy.abs())
    for k, parts in enumerate(rows):
        if parts:
            x, fdv, dy, fv = (torch.cat(t) for t in zip(*parts))
            eA[k] += 4 * fdv.max() * x.sum(0)[:, None]
            eB[k] += 4 * fv.max() * dy.sum(0)[None, :]
    dW = X.t() @ d if train_w else None
    eW = X.abs().t() @ ed + (c.n + 8) * U * (X.abs().t() @ d.abs()) if train_w else None
    return (dX, eX), list(zip(dA, eA)), list(zip(dB, eB)), (dW, eW)


def gate_backward(c, kind):
    """dG, dU in 64 bits from the stored 16-bit G, U and dH, with bounds of the rounded values."""
    h = half_step(c.dtype)
    g, u, dh = c.proj[0]["G"].double(), c.proj[1]["G"].double(), c.dY.double()
    a, slope = act(kind, g)
    floor = 2.0 ** -25 if c.dtype == torch.float16 else 0.0
    dg, du = dh * u * slope, dh * a
    if c.n <= 128 and c.n * c.h_out <= 2 ** 18:
        h = h * h
    eg = h * dg.abs() + 2.0 ** -20 * (dh * u).abs() * 1.13 * (1 + g.abs()) + floor
    eu = h * du.abs() + 2.0 ** -20 * (dh * g).abs() + floor
    return (dg, eg), (du, eu)


def check(got, ref, bound, dtype, what, rounded=False):
    """|got - ref| within the bound of the unrounded sum plus the output's rounding (unless `rounded`:
    the bound has it), elementwise; the smallest denormals' half step is the floor."""
    h = half_step(dtype)
    full = bound if rounded else bound + h * (ref.abs() + bound)
    full = full + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite values"
    bad = err > full
    if bad.any():
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements out of bound, first at {at}: got "
                             f"{float(got[at])!r}, want {float(ref[at])!r}, bound {float(full[at])!r}; worst "
                             f"err / bound {float((err / full).max()):.3g}")
