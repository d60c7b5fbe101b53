"""Arguments that lie in one wider array: column ranges that share no element are taken, whatever the
number of their rows; ranges that share one are refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    import gaussian_splatting_raster_b200 as P
    P.build()
    return P


def test_one_row_between_rows(P):
    """A single output row in the gap between the rows of an input."""
    w = torch.arange(24.0, device="cuda").reshape(4, 6)
    want = w.clone()
    want[1, 3:6] = w[2, 0:3] * 2
    P.lookup(w[:, :3], torch.tensor([2], dtype=torch.int32, device="cuda"), w[1:2, 3:6], scale=2.0)
    assert torch.equal(w, want)
    one = torch.ones(3, 3, device="cuda")
    y = torch.empty(1, 3, device="cuda")
    P.ffn(w[2:3, :3], None, one, one, y)
    P.ffn(w[2:3, :3], None, one, one, w[3:4, 3:6])
    assert torch.equal(w[3, 3:6], y[0])


def test_one_row_shared(P):
    w = torch.arange(24.0, device="cuda").reshape(4, 6)
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out in (w[1:2, 2:5], w[0:1, 0:3], w.view(-1)[4:7].view(1, 3), w.view(-1)[-7:-4].view(1, 3)):
        with pytest.raises(P.SplatError) as e:
            P.lookup(w[:, :3], ids, out)
        assert e.value.code == -1
    with pytest.raises(P.SplatError) as e:  # wider than the gap
        P.lookup(w.view(-1)[:24].view(4, 6)[:, :3], ids,
                 torch.as_strided(w, (1, 3), (6, 1), 5))
    assert e.value.code == -1
