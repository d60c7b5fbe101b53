"""Weight gradients of the feed-forward block over very many rows, where all terms of a sum have one sign:
what an accumulator loses by truncation adds up instead of averaging out.

Bounds, relative to the sum (u = R.U of the type): u for its rounding; the hidden values' own
roundings are independent, n of them, at most u each: 8 u / sqrt n; the accumulator holds at most
8,192 rows (bf16: 65,536), added 16 at a time by two truncations (of the products' sum, and of the
addition) that lose less than a unit in its last place each, 2^-22 of what it holds, which on average
is half of the whole: 8192 / 16 / 2 * 2^-22 = 2^-14 (2^-11), u / 8; the sums of those are fp32,
M / 8192 + 148 of them at most.
The mean of (got - exact) / exact has the last two, and of the roundings u / sqrt(3 F), taken five
times: the sums of one hidden unit lie closer to one another than the type's steps (their inputs are
averages over all rows), so only units round independently."""
import math

import pytest
import torch

import rows_util as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    import gaussian_splatting_raster_b200 as P
    P.build()
    return P


def _exact(x, wg, wu, wd, dy, act):
    x0, dy0 = x, dy
    wu, wd = wu.double(), wd.double()
    out = [torch.zeros_like(wu), torch.zeros_like(wu), torch.zeros_like(wd)]
    for r in range(0, x0.shape[0], 100000):
        x, dy = x0[r:r + 100000].double(), dy0[r:r + 100000].double()
        u = x @ wu.T
        a = u if wg is None else x @ wg.double().T
        if act == "silu":
            s = torch.sigmoid(a)
            f, d = a * s, s * (1 + a * (1 - s))
        else:
            c = 0.5 * torch.special.erfc(-a / math.sqrt(2))
            f, d = a * c, c + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        dh = dy @ wd
        out[2] += dy.T @ (f if wg is None else f * u)
        if wg is None:
            out[1] += (dh * d).T @ x
        else:
            out[0] += (dh * u * d).T @ x
            out[1] += (dh * f).T @ x
    return out


CASES = [  # M, D, F, O, gated, act
    (2_000_000, 16, 1024, 16, True, "silu"), (1_200_000, 4, 1024, 8, True, "gelu"),
    (5_000_000, 33, 64, 16, False, "gelu"), (1_500_000, 20, 32, 100, True, "silu")]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_sums_of_one_sign(P, case, dt):
    M, D, F, O, gated, act = case
    g = torch.Generator(device="cuda").manual_seed(M + F)

    def some(n, c, scale):
        return (torch.rand((n, c), generator=g, device="cuda") + 0.5).mul_(scale).to(dt)

    x, dy = some(M, D, 1.0), some(M, O, 2.0 ** -12)
    wg, wu, wd = some(F, D, 1 / D) if gated else None, some(F, D, 1 / D), some(O, F, 0.5)
    got = [torch.empty_like(wu), torch.empty_like(wu), torch.empty_like(wd)]
    P.ffn_backward(dy, x, wg, wu, wd, dw_gate=got[0] if gated else None, dw_up=got[1],
                   dw_down=got[2], act=act)
    P.rows_status()
    u = R.U[dt]
    held = 0.0 if dt == torch.float32 else 8 * u / math.sqrt(M)
    # (fp32: 8,192 additions, each rounded: 2^-24 sqrt(8192) of the sum, taken eight times)
    kept = u / 8 if dt != torch.float32 else 8 * 2.0 ** -24 * math.sqrt(8192)
    kept += (M / 8192 + 148) * R.U32
    for name, a, b in zip(("dw_gate", "dw_up", "dw_down"), got,
                          _exact(x, wg, wu, wd, dy, act)):
        if name == "dw_gate" and not gated:
            continue
        assert torch.isfinite(a).all()
        rel = (a.double() - b) / b
        worst, mean = rel.abs().max().item(), rel.mean().abs().item()
        assert worst <= u + held + kept, f"{name}: {worst:.3g}"
        assert mean <= held + kept + 5 * u / math.sqrt(3 * F), f"{name}: mean {mean:.3g}"
