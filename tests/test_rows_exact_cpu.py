"""What the exact cases can see: each tile of rows left out of a sum changes results after their rounding."""
import pytest
import torch

import rows_exact as E

TILE = 128  # rows of a tile on the tensor cores; the fp32 lanes' tiles are its multiples or halves


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("case", [c for c in E.FFNS if 128 < c[0] <= 60000], ids=str)
def test_a_tile_left_out_shows(case, dt):
    M, D, F, O, gated, _ = case
    x, wg, wu, wd, dy = E.ffn_inputs(M, D, F, O, gated, M + D)
    whole = E.ffn_results(x, wg, wu, wd, dy)
    for t in (x, wg, wu, wd, dy):  # inputs are what they are in every type
        assert t is None or torch.equal(t.to(dt).double(), t)
    names = [n for n in whole if n.startswith("dw")]
    for r in range(0, M, TILE):
        part = E.ffn_results(x[r:r + TILE], wg, wu, wd, dy[r:r + TILE])
        for n in names:
            assert not torch.equal((whole[n] - part[n]).to(dt), whole[n].to(dt)), (r, n)
            assert not torch.equal((whole[n] + part[n]).to(dt), whole[n].to(dt)), (r, n)


@pytest.mark.parametrize("case", E.LOOKUPS, ids=str)
def test_an_entry_left_out_shows(case):
    """In fp32 every entry, by itself: it is one of the sums' ones."""
    N, M, C, kind = case
    ids, dout = E.lookup_inputs(N, M, C, kind, M + N)
    sums = torch.zeros(N, C, dtype=torch.float64).index_add_(0, ids.long(), dout)
    assert sums.abs().max() < 2 ** 24 and (dout.abs() == 1).all()
    assert torch.equal(sums.float().double(), sums)
