"""Activations of the feed-forward block far out, where a result has few units to hide behind: each
value by itself, against 64 bits, with bounds relative to it.

Every block here passes one hidden value a column to its output: x has one column that is not zero,
the weights are ones and an identity, so a = x exactly, y = act(a) and, from dy with one 1 a row,
dx = act'(a); sums add zeros.

Bounds. u = R.U of the type, U32 = 2^-24.
  result and, above 128 rows, hidden value rounded to the type: 2 u, and its smallest step (half of it
  twice); powers below 2^-126 are zero: 2^-126 (1 + |a|) + 2^-126 |a|.
  silu: the exponent a log2 e is off by 2 U32 |a log2 e|, so a power by that times ln 2: 2 |a| U32.
  Powers and reciprocals are off by 2^-22 = 4 U32 each (the special function unit; expf and a
  division are nearer), products and sums by U32 each: (16 + 2 |a|) U32 of the value. The slope is
  s (1 + a (1 - s)), its error that of s (1 + |a| (1 - s)). Where e^-a overflows (-a > 88.7) the
  fp32 lanes give zero for |a| e^a < 2^-121.
  gelu, fp32 lanes: Phi(-|a|) = r P(r) e^{-a^2/2}, r = 1 / (1 + c |a|). r is off by 3 U32 (argument,
  reciprocal) and moves r P(r) by no more than its share; P is off by 0.2 U32 from the function and
  by 2 U32 from its last steps' roundings; the power 4 U32 and the exponent a^2 / 2 twice U32 of
  itself, two products U32 each: (12 + 2 a^2) U32 of Phi(-|a|), and U32 of 1 - Phi(-|a|). The value
  6 U32 more. The slope adds a phi(a): (8 + a^2) U32 of |a| phi.
  gelu, tensor cores: Phi by the published formula (Abramowitz and Stegun 7.1.26), whose own error is
  taken in 64 bits; e^{-a^2/2} as above, (24 + a^2) U32 of Phi(-|a|) and 2 U32 of Phi.
"""
import math

import pytest
import torch

import rows_util as R

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
VALUES = [-6e4, -1e4, -1e3, -300.0, -120.0, -90.0, -88.0, -86.0, -60.0, -40.0, -30.0, -23.0,
          -22.0, -21.5, -21.25, -21.0, -20.0, -15.0, -12.0, -9.0, -7.0, -5.5, -5.0, -4.0, -3.0,
          -2.0, -1.25, -1.0, -0.5, -1e-3, 0.0, 1e-3, 0.5, 1.0, 3.0, 5.0, 9.0, 21.5, 60.0, 300.0, 6e4]
BEYOND = [-3e38, -1e30, -1e6, 1e6, 1e30]  # not in fp16


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    import gaussian_splatting_raster_b200 as P
    P.build()
    return P


def _phi(a):
    """The normal distribution function. (1 + erf, and torch.special.ndtr, give zero at -9.)"""
    return 0.5 * torch.special.erfc(-a / math.sqrt(2))


def _expected(a, kind, dt, tensor):
    """(value, bound) of act(a) and act'(a); tensor: by the tensor-core kernels."""
    m = a.abs()
    if kind == "silu":
        s = torch.sigmoid(a)
        n = torch.sigmoid(-a)
        v, d = a * s, s + a * s * n
        ev = (16 + 2 * m) * R.U32 * v.abs()
        ed = (16 + 2 * m) * R.U32 * s * (1 + m * n)
    else:
        phi = torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        cdf, tail = _phi(a), _phi(-m)
        v, d = a * cdf, cdf + a * phi
        if tensor:
            z = m / math.sqrt(2)
            r = 1 / (1 + 0.3275911 * z)
            q = 0.5 * r * (0.254829592 + r * (-0.284496736 + r * (1.421413741 + r * (
                -1.453152027 + r * 1.061405429)))) * torch.exp(-z * z)
            ec = (q - tail).abs() + (24 + a * a) * R.U32 * tail + 2 * R.U32 * cdf
        else:
            ec = (12 + 2 * a * a) * R.U32 * tail + R.U32 * cdf
        ev = m * ec + 6 * R.U32 * v.abs()
        ed = ec + (8 + a * a) * R.U32 * m * phi + 2 * R.U32 * d.abs()
    flush = 2.0 ** -126 * (1 + 2 * m)
    if kind == "silu" and not tensor:
        flush = 2.0 ** -121
    return [(t, e + flush + 2 * R.U[dt] * (t.abs() + e) + R.TINY[dt]) for t, e in
            ((v, ev), (d, ed))]


SHAPES = [  # D, F, O, gated: one unit; hidden values in twice the bits; a plain block; both gated
    (1, 1, 1, False), (8, 32, 16, False), (8, 64, 64, False), (1, 1, 1, True), (16, 64, 64, True)]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("M", [39, 200, 3000])
def test_activation_alone(P, M, shape, kind, dt):
    D, F, O, gated = shape
    vals = VALUES + (BEYOND if dt != torch.float16 else [])
    a = torch.tensor(vals, dtype=torch.float64).repeat(-(-M // len(vals)))[:M].to(dt)
    x = torch.zeros(M, D, dtype=dt)
    x[:, 0] = a
    wu, wd = torch.zeros(F, D, dtype=dt), torch.zeros(O, F, dtype=dt)
    wu[:, 0] = 1
    wg = None
    if gated:  # u = 1 from a column of ones (or, with one column, from x itself: u = a)
        wg, wu = wu, wu.clone()
        if D > 1:
            x[:, 1] = 1
            wu[:, 0], wu[:, 1] = 0, 1
    unit = torch.arange(M) % min(F, O)
    n = min(F, O)
    wd[torch.arange(n), torch.arange(n)] = 1
    dy = torch.zeros(M, O, dtype=dt)
    dy[torch.arange(M), unit] = 1
    w = [None if t is None else t.cuda() for t in (wg, wu, wd)]
    y = torch.empty(M, O, dtype=dt, device="cuda")
    P.ffn(x.cuda(), *w, y, act=kind)
    a = a.double()
    tensor = dt != torch.float32
    scale = a if gated and D == 1 else torch.ones_like(a)
    v, e = _expected(a, kind, dt, tensor and M > 128)[0]
    # with u = a the product may leave fp16 (or even fp32): those rows are not what is asked here
    fits = (v * scale).abs() < torch.finfo(dt).max / 2
    assert fits.sum() > M // 2
    v, e = v * scale, (e + 2 * R.U32 * v.abs()) * scale.abs() + R.TINY[dt]
    R.close(y[:, :n].cpu()[fits], (v[fits, None].expand(-1, n), e[fits, None].expand(-1, n)), "y")
    if gated and D == 1:
        return
    dx = torch.empty(M, D, dtype=dt, device="cuda")
    P.ffn_backward(dy.cuda(), x.cuda(), *w, dx=dx, act=kind)
    R.close(dx[:, 0], _expected(a, kind, dt, tensor)[1], "dx")


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M", [3, 200])
def test_no_number_stays_with_its_row(P, M, kind, dt):
    """Rows of NaN, and of infinities of either sign, give rows that are not finite; rows beside
    them, far out on the left, are as they are without them."""
    D, F, O = 8, 64, 64
    g = torch.Generator().manual_seed(3)
    w = [(torch.rand(s, generator=g) + 0.1).to(dt).cuda() for s in ((F, D), (O, F))]
    x = torch.full((M, D), -30.0).to(dt)
    y, z = (torch.empty(M, O, dtype=dt, device="cuda") for _ in range(2))
    P.ffn(x.cuda(), None, *w, y, act=kind)
    for bad in (float("nan"), float("inf"), -float("inf")):
        b = x.clone()
        b[1, 2] = bad
        P.ffn(b.cuda(), None, *w, z, act=kind)
        assert not torch.isfinite(z[1]).any()
        assert torch.equal(z[0], y[0]) and torch.equal(z[2:], y[2:])
