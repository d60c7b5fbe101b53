"""Per-row operators where every result is exact: equal to the bit, in every type and kernel."""
import pytest
import torch

import rows_exact as E

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    import gaussian_splatting_raster_b200 as P
    P.build()
    return P


def _view(t, dt, pad):
    w = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=dt, device="cuda")
    w[:, :t.shape[1]] = t.to(dt).cuda()
    return w[:, :t.shape[1]]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("case", E.FFNS, ids=str)
def test_ffn(P, case, act, dt):
    M, D, F, O, gated, pad = case
    x, wg, wu, wd, dy = E.ffn_inputs(M, D, F, O, gated, M + D)
    want = E.ffn_results(x, wg, wu, wd, dy)
    xv, dyv = _view(x, dt, pad), _view(dy, dt, pad)
    w = [None if t is None else t.to(dt).cuda() for t in (wg, wu, wd)]
    got = {k: torch.full(v.shape, 7.0, dtype=dt, device="cuda") for k, v in want.items()}
    P.ffn(xv, *w, got["y"], act=act)
    P.ffn_backward(dyv, xv, *w, act=act, **{k: v for k, v in got.items() if k != "y"})
    for k, v in want.items():
        assert torch.equal(got[k].cpu(), v.to(dt)), k


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("case", E.LOOKUPS, ids=str)
def test_lookup_backward(P, case, dt):
    N, M, C, kind = case
    ids, dout = E.lookup_inputs(N, M, C, kind, M + N)
    want = torch.zeros(N, C, dtype=torch.float64).index_add_(0, ids.long(), dout) * 2
    got = torch.full((N, C), 7.0, dtype=dt, device="cuda")
    P.lookup_backward(dout.to(dt).cuda(), ids.cuda(), got, scale=2.0)
    assert torch.equal(got.cpu(), want.to(dt))


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("case", E.LOOKUPS, ids=str)
def test_lookup(P, case, dt):
    N, M, C, kind = case
    ids, _ = E.lookup_inputs(N, M, C, kind, M + N)
    table = torch.randint(-128, 129, (N, C), generator=torch.Generator().manual_seed(N)).to(dt)
    got = torch.full((M, C), 7.0, dtype=dt, device="cuda")
    P.lookup(table.cuda(), ids.cuda(), got, scale=-4.0)
    assert torch.equal(got.cpu(), table[ids.long()] * -4)
