"""Layer norm of constant and nearly constant rows far from zero, at widths on both sides of those whose rows are read again.

Bounds, with u = 2^-24 and D the additions one after another of a wide row's sum (8 of an eight, one an eight of a lane, 22 to join):
* a first mean is off by at most e0 = (D + 2) u |v|.  Of a constant row v the differences v - mean are exact and all alike, and
  their mean is off by (D + 2) u e0 at most, which is below 2^-26 |v| for every width: half a step of fp32 around v is
  2^-25 |v| or more, so the corrected mean is v itself, and Y is beta.
* the variance about the corrected mean is off by 3 (D + 8) u (var + e0^2): two sums and a difference of theirs.
* where the row is not constant the mean is rounded once, u |mean|, and off by the correction's (D + 2) u e0 besides."""
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests.test_gpu_norm import DT, check

pytestmark = pytest.mark.gpu

u, EPS = 2.0 ** -24, 1e-5
WIDTHS = [4096, 24576, 24584, 65544, 100008, 131064, 1 << 20]


def depth(w):
    return 30 + -(-w // 8192)


def first_error(w, v):
    return (depth(w) + 2) * u * v


def forward(X, gamma, beta):
    n, w = X.shape
    Y = torch.full_like(X, float("nan"))
    mean, rstd = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    sg.sgmv_layer_norm_apply(X, gamma, beta, Y, EPS, mean=mean, rstd=rstd)
    return Y, mean, rstd


def parameters(w, dtype):
    g = torch.Generator().manual_seed(w)
    return [t.to(dtype).cuda() for t in (1 + 0.3 * torch.randn(w, generator=g), torch.randn(w, generator=g))]


def values(n, dtype):
    """n values from 1 to 65504 of either sign, spread over their logarithm."""
    v = torch.logspace(0, 4.8163, n, dtype=torch.float64).clamp(max=65504.0).to(dtype)
    return torch.where(torch.arange(n) % 3 == 2, -v, v)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("w", WIDTHS)
def test_constant_rows(w, dtype):
    n = 200 if w < 1 << 20 else 60
    gamma, beta = parameters(w, DT[dtype])
    v = values(n, DT[dtype]).cuda()
    Y, mean, rstd = forward(v[:, None].expand(n, w).contiguous(), gamma, beta)
    assert torch.equal(mean, v.float())
    assert torch.equal(Y, beta.expand(n, w))
    e0 = first_error(w, v.double().abs())
    ev = 3 * (depth(w) + 8) * u * e0 * e0
    low, high = (EPS + ev) ** -0.5, (EPS - ev).clamp(min=1e-30) ** -0.5
    assert (rstd.double() >= low * (1 - 6 * u)).all() and (rstd.double() <= high * (1 + 6 * u)).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("w", [24584, 65544, 100008, 131064, 1 << 20])
def test_nearly_constant_rows(w, dtype):
    """One value in about a hundred is a step of the format higher."""
    n, dt = 24, DT[dtype]
    gamma, beta = parameters(w, dt)
    v = values(n, dt).float().abs()
    up = torch.rand(n, w, generator=torch.Generator().manual_seed(w + 1)) < 0.01
    step = torch.finfo(dt).eps * 2.0 ** torch.floor(torch.log2(v))
    X = (v[:, None] + torch.where(up, 1.0, 0.0) * step[:, None]).clamp(max=65504.0).to(dt).cuda()
    Y, mean, rstd = forward(X, gamma, beta)
    x = X.double()
    m = x.mean(1)
    d = x - m[:, None]
    var = (d * d).mean(1)
    e0 = first_error(w, x.abs().amax(1))
    em = u * m.abs() + (depth(w) + 2) * u * e0
    check(mean, m, em, "mean")
    ev = 3 * (depth(w) + 8) * u * (var + e0 * e0)
    er = 0.5 * ev / (var + EPS) / (1 - ev / (var + EPS)).clamp(min=0.1) + 6 * u
    r = (var + EPS) ** -0.5
    check(rstd, r, r * er, "rstd")
    g, b = gamma.double(), beta.double()
    y = d * r[:, None] * g + b
    ey = g.abs() * r[:, None] * (em[:, None] + (d.abs() + em[:, None]) * (er[:, None] + 5 * u)) + 2 * u * (b.abs() + y.abs())
    check(Y, y, ey, "Y")


@pytest.mark.parametrize("w", [4096, 24584, 100008])
def test_sums_beyond_fp32(w):
    """A row whose sum leaves fp32, with and without infinities in it, has a mean of infinity; the others are as they were."""
    gamma, beta = parameters(w, torch.bfloat16)
    X = torch.randn(7, w, generator=torch.Generator().manual_seed(w)).bfloat16().cuda()
    clean = forward(X, gamma, beta)
    X[1], X[4], X[5, 3] = 3e38, -3e38, float("inf")
    got = forward(X, gamma, beta)
    assert torch.equal(got[1][[1, 4, 5]], torch.tensor([float("inf"), -float("inf"), float("inf")], device="cuda"))
    for a, b in zip(got, clean):
        assert torch.equal(a[[0, 2, 3, 6]], b[[0, 2, 3, 6]])
    assert got[0][[1, 4, 5]].isnan().any(1).all()
