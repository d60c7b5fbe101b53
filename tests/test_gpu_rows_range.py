"""Gradients of fp16 blocks far from 1: as of a mean over very many rows, where dy and what it makes of
the hidden values' gradients lie at fp16's smallest steps, and large ones.

Expected values and bounds are those of the same gradients times a power of two that brings the largest
|dy| into [2^-6, 16), where the reference's bounds hold, scaled back; results are rounded to fp16
once more (half of its smallest step, 2^-25). Where the sizes of x and the weights would carry hidden
values themselves out of the range there is nothing to expect."""
import pytest
import torch

import rows_util as R

pytestmark = pytest.mark.gpu
H = torch.float16


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    import gaussian_splatting_raster_b200 as P
    P.build()
    return P


def _inputs(M, D, F, O, gated, seed, dy_size, wd_size):
    g = torch.Generator().manual_seed(seed)
    x = (torch.rand(M, D, generator=g) + 0.5).to(H)
    wg, wu = ((torch.rand(F, D, generator=g) / D).to(H) for _ in range(2))
    wd = ((torch.rand(O, F, generator=g) + 0.5) * wd_size).to(H)
    dy = ((torch.rand(M, O, generator=g) + 0.25) * dy_size).to(H)
    return x, wg if gated else None, wu, wd, dy


def _run(P, x, wg, wu, wd, dy, act):
    c = [None if t is None else t.cuda() for t in (x, wg, wu, wd)]
    out = dict(dx=torch.empty_like(c[0]), dw_up=torch.empty_like(c[2]),
               dw_down=torch.empty_like(c[3]))
    if wg is not None:
        out["dw_gate"] = torch.empty_like(c[1])
    P.ffn_backward(dy.cuda(), *c, act=act, **out)
    P.rows_status()
    return out


CASES = [  # M, D, F, O, gated, act, |dy|, |wd|
    (20000, 24, 128, 32, True, "silu", 2.0 ** -20, 2.0 ** -12),
    (20000, 24, 128, 32, False, "gelu", 2.0 ** -23, 2.0 ** -10),
    (20000, 9, 30, 5, True, "gelu", 2.0 ** -20, 2.0 ** -9),
    (300, 33, 70, 17, True, "silu", 2.0 ** -16, 2.0 ** -8),
    (3000, 120, 40, 32, True, "silu", 3e4, 0.25), (300, 60, 6, 5, False, "gelu", 6e3, 8.0)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_far_from_one(P, case):
    M, D, F, O, gated, act, size, wd_size = case
    x, wg, wu, wd, dy = _inputs(M, D, F, O, gated, M + F, size, wd_size)
    out = _run(P, x, wg, wu, wd, dy, act)
    k = 2.0 ** (-3 if size < 1 else 0) / 2.0 ** round(torch.log2(dy.double().max()).item())
    ref = R.ffn_ref(x, wg, wu, wd, act, dy.double() * k)
    for name, got in out.items():
        v, e = ref[name]
        v, e = v / k, e / k
        if name == "dw_down":  # of the hidden values, which are not scaled
            v0, e0 = R.ffn_ref(x, wg, wu, wd, act, dy)[name]
            v, e = v0, e0
        fits = v.abs() < 6e4  # (weights' sums of the large cases do not)
        assert fits.all() if name == "dx" or size < 1 else True, name
        if not fits.any():
            continue
        R.close(got.cpu()[fits], (v[fits], (e + 2.0 ** -25)[fits]), name)
        assert (got.cpu()[fits] != 0).float().mean() > 0.9 or (v.abs() < 2.0 ** -24).any(), name


@pytest.mark.parametrize("gated", [True, False])
def test_powers_of_two_pass_through(P, gated):
    """Two calls whose dy differ by a power of two, both small enough to be scaled to the same values:
    their results differ by that power, bit by bit, where they have all their digits."""
    x, wg, wu, wd, dy = _inputs(2000, 24, 128, 32, gated, 5, 1.0, 1.0)
    a = _run(P, x, wg, wu, wd, (dy * 2.0 ** -7).to(H), "gelu")
    b = _run(P, x, wg, wu, wd, (dy * 2.0 ** -9).to(H), "gelu")
    for k in a:
        full = b[k].abs() >= 2.0 ** -13
        assert full.float().mean() > 0.5
        if k != "dw_down":
            assert torch.equal(a[k][full], (b[k].float() * 4).to(H)[full]), k


def test_one_row_does_not_scale_the_others_away(P):
    """A row of infinities or NaN in dy leaves the other rows' dx as they are without it."""
    x, wg, wu, wd, dy = _inputs(700, 24, 128, 32, True, 6, 2.0 ** -20, 2.0 ** -10)
    dy[3] = 0
    want = _run(P, x, wg, wu, wd, dy, "silu")["dx"]
    for bad in (float("inf"), float("nan")):
        d = dy.clone()
        d[3] = bad
        got = _run(P, x, wg, wu, wd, d, "silu")["dx"]
        assert not torch.isfinite(got[3]).any()
        assert torch.equal(got[:3], want[:3]) and torch.equal(got[4:], want[4:])
