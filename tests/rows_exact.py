"""Inputs of the per-row operators whose results are whole numbers that no step rounds, so that a result
is right to the bit or wrong: a tile, a split, a chunk or an entry left out or taken twice shows, however
long the sums are.

Feed-forward block: x is 1 or 2; a unit's gate is 32 times one column of x, so a is 32 or 64, where
both activations are a itself and their slopes 1, in fp32 (e^-32 is below half a step of 1); u is plus or
minus a column. Hidden values are at most 128, da and du at most 128, all with few bits; sums stay below
2^24. Without a gate h = a."""
import torch


def ffn_inputs(M, D, F, O, gated, seed):
    """x, wg, wu, wd, dy in 64 bits."""
    g = torch.Generator().manual_seed(seed)

    def sign(*s):
        return torch.randint(0, 2, s, generator=g).double() * 2 - 1

    x = torch.randint(1, 3, (M, D), generator=g).double()
    f = torch.arange(F)
    big = torch.zeros(F, D, dtype=torch.float64)
    big[f, f % D] = 32
    wu = torch.zeros(F, D, dtype=torch.float64)
    wu[f, (7 * f + 3) % D] = sign(F)
    wd = torch.zeros(O, F, dtype=torch.float64)
    wd[f % O, f] = sign(F)
    wd[(3 * f + 1) % O, f] = sign(F)
    dy = sign(M, O)
    return (x, big, wu, wd, dy) if gated else (x, None, big, wd, dy)


def ffn_results(x, wg, wu, wd, dy):
    u = x @ wu.T
    a = u if wg is None else x @ wg.T
    assert (a >= 32).all()
    h = a if wg is None else a * u
    dh = dy @ wd
    out = dict(y=h @ wd.T, dw_down=dy.T @ h)
    if wg is None:
        out.update(dx=dh @ wu, dw_up=dh.T @ x)
    else:
        da, du = dh * u, dh * a
        out.update(dx=da @ wg + du @ wu, dw_gate=da.T @ x, dw_up=du.T @ x)
    return out


FFNS = [  # M, D, F, O, gated, pad
    (1, 5, 40, 7, True, 0), (129, 57, 64, 64, True, 0), (300, 128, 1000, 3, True, 0),
    (5001, 57, 700, 64, True, 3), (12000, 3, 33, 5, True, 8), (40000, 57, 64, 64, True, 0),
    (40000, 128, 200, 128, True, 0), (40000, 100, 64, 20, False, 0),
    (60000, 128, 60, 40, True, 0), (60000, 35, 128, 48, True, 3), (40000, 33, 520, 33, False, 1),
    (20000, 128, 32, 100, False, 1), (20000, 3, 1000, 9, False, 0),
    (65000, 9, 300, 11, True, 0),
    # several launches of the weight gradients: 9 splits, and 4, of 8,192 rows
    (160000, 8, 1024, 16, True, 0), (100000, 4, 1024, 8, True, 0),
    # ... the last of them with fewer tiles than splits
    (9 * 8192 + 1, 9, 1024, 11, True, 3), (9 * 8192 + 300, 9, 1024, 11, True, 0),
    (2 * 4 * 8192 + 130, 4, 1024, 8, True, 1)]


def lookup_inputs(N, M, C, kind, seed):
    """ids and dout of plus and minus ones."""
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(M, generator=g, dtype=torch.float64)
    ids = {"uniform": u * N, "skewed": u ** 6 * N, "same": u * 0,
           "sorted": torch.arange(M) * (N / M)}[kind].int()
    return ids, torch.randint(0, 2, (M, C), generator=g).double() * 2 - 1


LOOKUPS = [  # N, M, C, ids
    (1, 70000, 4, "same"), (3, 50001, 33, "skewed"), (500, 300000, 16, "uniform"),
    (19, 2047, 8, "skewed"), (70000, 200000, 19, "uniform"), (1000, 100000, 48, "sorted"),
    (400000, 150000, 3, "uniform"), (2, 1500000, 5, "skewed")]
