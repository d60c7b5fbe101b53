"""Per-row operators on the GPU (through the binding and the C ABI) against 64-bit references with
the rounding bounds of rows_util."""
import ctypes

import numpy as np
import pytest
import torch

import rows_util as R

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    import gaussian_splatting_raster_b200 as P
    P.build()
    P.load_library()
    return P


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _view(t, pad, lead=0):
    """t as a column range of a wider CUDA tensor filled with NaN, and the wide tensor."""
    if pad == 0 and lead == 0:
        w = t.cuda()
        return w, w
    w = torch.full((t.shape[0], lead + t.shape[1] + pad), float("nan"), dtype=t.dtype,
                   device="cuda")
    w[:, lead:lead + t.shape[1]] = t.cuda()
    return w[:, lead:lead + t.shape[1]], w


def _out(rows, cols, dt, pad, lead=0):
    w = torch.full((rows, lead + cols + pad), 7.0, dtype=dt, device="cuda")
    return w[:, lead:lead + cols], w


def _untouched(w, lead, cols):
    assert (w[:, :lead] == 7).all() and (w[:, lead + cols:] == 7).all()


# -- lookup ---------------------------------------------------------------------------------------

def _ids(kind, M, N, g):
    if kind == "sorted":
        return torch.sort(torch.randint(0, N, (M,), generator=g)).values.int()
    if kind == "same":
        return torch.full((M,), N - 1, dtype=torch.int32)
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if kind == "outside":  # below, above, at both ends of int32
        ids = torch.randint(-2, N + 2, (M,), generator=g).int()
        ids[::5] = 2**31 - 1
        ids[1::7] = -2**31
        return ids
    if kind == "skewed":
        return (torch.rand(M, generator=g, dtype=torch.float64) ** 6 * N).int()
    if kind == "reverse":
        return torch.sort(torch.randint(0, N, (M,), generator=g), descending=True).values.int()
    return torch.randint(0, N, (M,), generator=g).int()


LOOKUPS = [  # N, M, C, ids, pad, lead
    (1, 1, 1, "uniform", 0, 0), (5, 3, 7, "uniform", 0, 0), (9, 40, 1, "skewed", 2, 1),
    (100, 257, 32, "uniform", 0, 0), (19, 1000, 33, "sorted", 3, 0), (7, 300, 64, "same", 0, 0),
    (7, 300, 5, "none", 0, 0), (64, 999, 24, "outside", 8, 8), (3, 5000, 48, "skewed", 0, 0),
    (1023, 3000, 16, "reverse", 0, 0), (1024, 3000, 19, "uniform", 5, 0),
    (70000, 20000, 8, "uniform", 0, 0), (1, 70000, 4, "uniform", 0, 0),
    (12, 40, 1025, "uniform", 0, 0), (4, 9, 8192, "uniform", 0, 0), (300, 9000, 128, "skewed", 1, 1),
    (2, 33000, 2, "uniform", 0, 0), (40, 2048, 8, "uniform", 0, 0), (40, 2049, 8, "skewed", 0, 0),
    (500000, 2047, 3, "outside", 0, 0), (50001, 3, 33, "uniform", 0, 0), (3, 1025, 60, "skewed", 4, 0),
    (60000, 20000, 20, "skewed", 0, 0), (60001, 30000, 11, "same", 0, 0),
    (60000, 2000, 130, "sorted", 0, 0), (100001, 40000, 3, "outside", 0, 0),
]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("case", LOOKUPS, ids=str)
def test_lookup(P, case, dt):
    N, M, C, kind, pad, lead = case
    g = _gen(N + M + C)
    table = torch.randn(N, C, generator=g).to(dt)
    ids = _ids(kind, M, N, g)
    t, _ = _view(table, pad, lead)
    out, wide = _out(M, C, dt, pad, lead)
    P.lookup(t, ids.cuda(), out, scale=1.7)
    R.close(out, R.lookup_ref(table, ids, float(np.float32(1.7))), "lookup")
    _untouched(wide, lead, C)


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("case", LOOKUPS, ids=str)
def test_lookup_backward(P, case, dt):
    N, M, C, kind, pad, lead = case
    g = _gen(N + M + C + 1)
    dout = torch.randn(M, C, generator=g).to(dt)
    ids = _ids(kind, M, N, g)
    d, _ = _view(dout, pad, lead)
    dt_, wide = _out(N, C, dt, pad, lead)
    P.lookup_backward(d, ids.cuda(), dt_, scale=0.3)
    R.close(dt_, R.lookup_grad_ref(dout, ids, N, float(np.float32(0.3))), "lookup_backward")
    _untouched(wide, lead, C)
    again = torch.empty((N, C), dtype=dt, device="cuda")
    P.lookup_backward(d, ids.cuda(), again, scale=0.3)
    assert torch.equal(again, dt_)  # the same bits on every run


def test_lookup_large(P):
    """More than 2^31 elements in the output and the gradient's input, three sort passes."""
    N, M, C = 1_100_000, 17_000_000, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(-1, N, (M,), generator=g, device="cuda").int()
    table = torch.randn(N, C, generator=g, device="cuda").bfloat16()
    out = torch.empty((M, C), dtype=torch.bfloat16, device="cuda")
    P.lookup(table, ids, out, scale=2.0)
    for r in (0, M // 2, M - 5000):
        i = ids[r:r + 5000].long()
        want = torch.where((i >= 0)[:, None], table[i.clamp_min(0)] * 2, 0)  # exact in bf16
        assert torch.equal(out[r:r + 5000], want)
    dtable = torch.empty((N, C), dtype=torch.bfloat16, device="cuda")
    P.lookup_backward(out, ids, dtable)
    sel = torch.cat([torch.arange(20), torch.arange(N - 20, N), torch.randint(0, N, (24,))])
    for n in sel.tolist():
        rows = out[ids == n].double().cpu()
        ref = R.lookup_grad_ref(rows.bfloat16(), torch.zeros(rows.shape[0]), 1, 1.0)
        R.close(dtable[n:n + 1], ref, f"row {n}")


def test_lookup_special_values(P):
    """Infinities and NaN stay with their rows; rows without an id stay zero whatever the scale."""
    t = torch.tensor([[1.0, float("inf")], [float("nan"), -2.0], [0.5, -0.0]]).cuda()
    ids = torch.tensor([0, -1, 2, 1, 3], dtype=torch.int32).cuda()
    out = torch.full((5, 2), 9.0, device="cuda")
    P.lookup(t, ids, out, scale=float("inf"))
    o = out.cpu()
    assert o[0, 0] == float("inf") and o[0, 1] == float("inf")
    assert (o[1] == 0).all() and (o[4] == 0).all() and torch.isnan(o[3, 0])
    d = torch.ones(5, 2).cuda()
    d[1] = float("nan")  # masked: takes no part
    d[3, 0] = float("inf")
    g = torch.full((4, 2), 9.0, device="cuda")
    P.lookup_backward(d, ids, g, scale=2.0)
    assert torch.equal(g.cpu(), torch.tensor([[2.0, 2], [float("inf"), 2], [2, 2], [2, 2]]))


def test_lookup_empty(P):
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    P.lookup(torch.ones(3, 4, device="cuda"), z, torch.empty(0, 4, device="cuda"))
    g = torch.full((3, 4), 5.0, device="cuda")
    P.lookup_backward(torch.empty(0, 4, device="cuda"), z, g)
    assert (g == 0).all()
    P.lookup_backward(torch.ones(2, 4, device="cuda"), torch.zeros(2, dtype=torch.int32).cuda(),
                      torch.empty(0, 4, device="cuda"))
    out = torch.full((2, 4), 5.0, device="cuda")
    P.lookup(torch.empty(0, 4, device="cuda"), torch.zeros(2, dtype=torch.int32).cuda(), out)
    assert (out == 0).all()


def test_lookup_broadcast_rows(P):
    """One gradient row for all (stride 0), and output columns between a neighbour's."""
    ids = torch.tensor([1, 0, 1, 1], dtype=torch.int32).cuda()
    d = torch.tensor([[1.0, 2.0, 3.0]]).cuda().expand(4, 3)
    wide = torch.full((2, 6), 7.0, device="cuda")
    P.lookup_backward(d, ids, wide[:, 3:])
    assert torch.equal(wide.cpu(), torch.tensor([[7.0, 7, 7, 1, 2, 3], [7, 7, 7, 3, 6, 9]]))
    buf = torch.full((2, 6), 7.0, device="cuda")
    src = torch.arange(6.0).cuda().reshape(2, 3)
    P.lookup(src, torch.tensor([1, 0], dtype=torch.int32).cuda(), buf[:, 3:])
    assert torch.equal(buf.cpu(), torch.tensor([[7.0, 7, 7, 3, 4, 5], [7, 7, 7, 0, 1, 2]]))
    # from one half of the same array into the other
    buf[:, :3] = src
    P.lookup(buf[:, :3], torch.tensor([1, 1], dtype=torch.int32).cuda(), buf[:, 3:])
    assert torch.equal(buf.cpu(), torch.tensor([[0.0, 1, 2, 3, 4, 5], [3, 4, 5, 3, 4, 5]]))


# -- feed-forward block ---------------------------------------------------------------------------

FFNS = [  # M, D, F, O, gated, act, pad
    (1, 1, 1, 1, True, "silu", 0), (1, 57, 256, 64, True, "gelu", 0), (2, 21, 33, 5, False, "gelu", 3),
    (7, 36, 100, 64, True, "silu", 0), (63, 12, 64, 1, False, "silu", 0),
    (64, 16, 65, 16, True, "gelu", 8), (65, 33, 63, 17, True, "silu", 1),
    (127, 64, 128, 64, False, "gelu", 0), (128, 128, 192, 128, True, "gelu", 0),
    (129, 127, 70, 127, True, "silu", 1), (300, 57, 256, 48, True, "gelu", 0),
    (1000, 65, 129, 66, False, "silu", 2), (1000, 8, 1024, 3, True, "silu", 0),
    (513, 128, 1024, 128, True, "silu", 0), (4097, 21, 40, 9, False, "gelu", 0),
    (20000, 30, 130, 62, True, "silu", 2), (40000, 57, 64, 64, True, "gelu", 0),
    # several row tiles a CTA at every combination of widths up to and above 64
    (40000, 128, 200, 128, True, "silu", 0), (40000, 100, 64, 20, False, "gelu", 0),
    (40000, 40, 70, 128, True, "silu", 0), (60000, 128, 60, 40, True, "gelu", 0),
    (40000, 33, 520, 33, False, "silu", 1), (30000, 128, 100, 128, False, "silu", 0),
    # chunks of units that a cluster cannot share evenly
    (5001, 57, 700, 64, True, "gelu", 3), (1500, 90, 449, 127, False, "silu", 1),
    (300, 128, 1000, 3, True, "silu", 0),
    # few inputs and outputs of many hidden units
    (700, 2, 104, 21, True, "gelu", 3), (20000, 3, 1000, 9, False, "silu", 0),
    (3000, 15, 70, 2, True, "silu", 0), (30000, 1, 1024, 1, True, "gelu", 0),
    # a few hidden units, few and many rows
    (200, 61, 1, 3, True, "silu", 8), (700, 128, 16, 128, True, "gelu", 0),
    (20000, 61, 1, 3, True, "silu", 8), (20000, 128, 32, 100, False, "gelu", 1),
    (20000, 70, 17, 64, True, "silu", 0), (12000, 3, 33, 5, True, "gelu", 8),
]


def _ffn_inputs(M, D, F, O, gated, dt, seed):
    g = _gen(seed)
    x = torch.randn(M, D, generator=g).to(dt)
    wg = (torch.randn(F, D, generator=g) / D ** 0.5).to(dt) if gated else None
    wu = (torch.randn(F, D, generator=g) / D ** 0.5).to(dt)
    wd = (torch.randn(O, F, generator=g) / F ** 0.5).to(dt)
    dy = torch.randn(M, O, generator=g).to(dt)
    return x, wg, wu, wd, dy


def _cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("case", FFNS, ids=str)
def test_ffn(P, case, dt):
    M, D, F, O, gated, act, pad = case
    x, wg, wu, wd, _ = _ffn_inputs(M, D, F, O, gated, dt, M + D)
    xv, _ = _view(x, pad, pad)
    y, wide = _out(M, O, dt, pad, pad)
    w = [_cuda(t) for t in (wg, wu, wd)]
    P.ffn(xv, *w, y, act=act)
    R.close(y, R.ffn_ref(x, wg, wu, wd, act)["y"], "y")
    _untouched(wide, pad, O)
    again = torch.empty((M, O), dtype=dt, device="cuda")
    P.ffn(xv, *w, again, act=act)
    assert torch.equal(again, y)


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("case", FFNS, ids=str)
def test_ffn_backward(P, case, dt):
    M, D, F, O, gated, act, pad = case
    x, wg, wu, wd, dy = _ffn_inputs(M, D, F, O, gated, dt, M + F)
    ref = R.ffn_ref(x, wg, wu, wd, act, dy)
    xv, _ = _view(x, pad, pad)
    dyv, _ = _view(dy, pad, pad)
    w = [_cuda(t) for t in (wg, wu, wd)]

    def run():
        dx, wide = _out(M, D, dt, pad, pad)
        o = dict(dx=dx, dw_up=torch.full((F, D), 7.0, dtype=dt, device="cuda"),
                 dw_down=torch.full((O, F), 7.0, dtype=dt, device="cuda"))
        if gated:
            o["dw_gate"] = torch.full((F, D), 7.0, dtype=dt, device="cuda")
        P.ffn_backward(dyv, xv, *w, act=act, **o)
        _untouched(wide, pad, D)
        return o

    a, b = run(), run()
    for k in a:
        R.close(a[k], ref[k], k)
        assert torch.equal(a[k], b[k]), k
    # each gradient alone is the same gradient
    for k in a:
        one = torch.full_like(a[k], 3.0)
        P.ffn_backward(dyv, xv, *w, act=act, **{k: one})
        assert torch.equal(one, a[k]), k


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False])
def test_ffn_gradient_equals_differences(P, act, gated):
    """<gradient, direction> against central differences of the 64-bit <dy, y>: the difference is
    off by eps^2 times third derivatives (1e-8 here), the kernel by its bound."""
    x, wg, wu, wd, dy = _ffn_inputs(40, 9, 20, 6, gated, torch.float32, 3)
    w = [_cuda(t) for t in (wg, wu, wd)]
    t = {"x": x, "wg": wg, "wu": wu, "wd": wd}
    names = {"x": "dx", "wg": "dw_gate", "wu": "dw_up", "wd": "dw_down"}
    got = {names[k]: torch.empty_like(v.cuda()) for k, v in t.items() if v is not None}
    P.ffn_backward(dy.cuda(), x.cuda(), *w, act=act, **got)
    bound = R.ffn_ref(x, wg, wu, wd, act, dy)
    R.U[torch.float64] = R.TINY[torch.float64] = 0.0
    t = {k: None if v is None else v.double() for k, v in t.items()}
    g = _gen(9)
    for k, v in t.items():
        if v is None:
            continue
        d = torch.randn(v.shape, generator=g, dtype=torch.float64)
        eps = 1e-5
        Lp, Lm = [(dy.double() * R.ffn_ref(*[a + s * eps * d if n == k else a
                                             for n, a in t.items()], act)["y"][0]).sum()
                  for s in (1, -1)]
        slack = (bound[names[k]][1] * d.abs()).sum() + 1e-6
        assert abs((Lp - Lm) / (2 * eps) - (got[names[k]].cpu().double() * d).sum()) <= slack


@pytest.mark.parametrize("dt", DTYPES, ids=str)
def test_ffn_rows_stay_apart(P, dt):
    """A row of NaN or infinities leaves every other row's result as it was, forward and dx, and
    the rows behind a partial tile add nothing to the weight gradients."""
    M, D, F, O = 200, 20, 70, 30
    x, wg, wu, wd, dy = _ffn_inputs(M, D, F, O, True, dt, 11)
    w = [_cuda(t) for t in (wg, wu, wd)]
    y0, y1 = (torch.empty(M, O, dtype=dt, device="cuda") for _ in range(2))
    d0, d1 = (torch.empty(M, D, dtype=dt, device="cuda") for _ in range(2))
    P.ffn(x.cuda(), *w, y0)
    P.ffn_backward(dy.cuda(), x.cuda(), *w, dx=d0)
    bad = x.clone()
    bad[3] = float("nan")
    bad[77, 5] = float("inf")
    P.ffn(bad.cuda(), *w, y1)
    P.ffn_backward(dy.cuda(), bad.cuda(), *w, dx=d1)
    keep = torch.ones(M, dtype=torch.bool)
    keep[[3, 77]] = False
    assert torch.equal(y0[keep.cuda()], y1[keep.cuda()]) and torch.isnan(y1[3]).all()
    assert torch.equal(d0[keep.cuda()], d1[keep.cuda()])


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_far_arguments(P, act, dt):
    """Arguments far out on both sides of the activation: no overflow on the way to a finite
    result."""
    v = torch.tensor([-300.0, -90.0, -60.0, -20.0, -8.0, -1e-3, 0.0, 1e-3, 8.0, 20.0, 60.0, 90.0,
                      300.0])
    x = v[:, None].to(dt)
    one = torch.ones(1, 1).to(dt)
    for M in (1, 40):
        xs = x.repeat(M, 1)
        y = torch.empty_like(xs.cuda())
        P.ffn(xs.cuda(), None, one.cuda(), one.cuda(), y, act=act)
        ref = R.ffn_ref(xs, None, one, one, act, torch.ones_like(xs))
        R.close(y, ref["y"], "y")
        dx = torch.empty_like(y)
        P.ffn_backward(torch.ones_like(y), xs.cuda(), None, one.cuda(), one.cuda(), dx=dx, act=act)
        R.close(dx, ref["dx"], "dx")


@pytest.mark.parametrize("dt", DTYPES, ids=str)
def test_ffn_empty(P, dt):
    w = torch.ones(5, 3, device="cuda", dtype=dt)
    wd = torch.ones(2, 5, device="cuda", dtype=dt)
    x, y = torch.empty(0, 3, device="cuda", dtype=dt), torch.empty(0, 2, device="cuda", dtype=dt)
    P.ffn(x, w, w, wd, y)
    g = [torch.full_like(w, 9), torch.full_like(w, 9), torch.full_like(wd, 9)]
    P.ffn_backward(y, x, w, w, wd, torch.empty_like(x), *g)
    assert all((t == 0).all() for t in g)
    P.ffn_backward(y, x, w, w, wd, dx=torch.empty_like(x))


@pytest.mark.parametrize("dt", DTYPES, ids=str)
def test_ffn_broadcast_row(P, dt):
    """One input row for all rows (stride 0): every row has the row's result, dx has every row."""
    x, wg, wu, wd, dy = _ffn_inputs(300, 24, 40, 16, True, dt, 4)
    w = [_cuda(t) for t in (wg, wu, wd)]
    xe = x[:1].expand(300, 24)
    y = torch.empty(300, 16, dtype=dt, device="cuda")
    P.ffn(xe[:1].cuda().expand(300, 24), *w, y)
    ref = R.ffn_ref(xe, wg, wu, wd, "silu", dy)
    R.close(y, ref["y"])
    dx = torch.empty(300, 24, dtype=dt, device="cuda")
    dw = torch.empty_like(w[1])
    P.ffn_backward(dy.cuda(), x[:1].cuda().expand(300, 24), *w, dx=dx, dw_up=dw)
    R.close(dx, ref["dx"])
    R.close(dw, ref["dw_up"])


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("shift", [1, 3, 8])
def test_ffn_rows_anywhere(P, dt, shift):
    """Arrays that start at an odd element, at the first and last elements of their allocation, with
    wide gaps between rows, and with rows that overlap one another (inputs)."""
    M, D, F, O = 700, 29, 66, 31
    x, wg, wu, wd, dy = _ffn_inputs(M, D, F, O, True, dt, 17)
    w = [_cuda(t) for t in (wg, wu, wd)]
    ref = R.ffn_ref(x, wg, wu, wd, "silu", dy)

    def strided(t, ld):
        flat = torch.full((shift + (M - 1) * ld + t.shape[1],), float("nan"), dtype=dt).cuda()
        v = flat[shift:].as_strided((M, t.shape[1]), (ld, 1), shift)
        v.copy_(t)
        return v

    for ldx, ldy in ((D, O), (D + 1, O + 3), (8 * D, 8 * O), (300, 301)):
        xv, dyv = strided(x, ldx), strided(dy, ldy)
        y = torch.empty(M, O, dtype=dt, device="cuda")
        P.ffn(xv, *w, y)
        R.close(y, ref["y"], "y")
        dx, dw = torch.empty(M, D, dtype=dt, device="cuda"), torch.empty_like(w[2])
        P.ffn_backward(dyv, xv, *w, dx=dx, dw_down=dw)
        R.close(dx, ref["dx"], "dx")
        R.close(dw, ref["dw_down"], "dw_down")
    g = _gen(3)
    flat = torch.randn(shift + (M - 1) * 5 + D, generator=g).to(dt)
    xo = flat.as_strided((M, D), (5, 1), shift)
    ref = R.ffn_ref(xo, wg, wu, wd, "gelu", dy)
    xv = flat.cuda().as_strided((M, D), (5, 1), shift)
    y = torch.empty(M, O, dtype=dt, device="cuda")
    P.ffn(xv, *w, y, act="gelu")
    R.close(y, ref["y"], "y")
    dw = torch.empty_like(w[0])
    P.ffn_backward(dy.cuda(), xv, *w, dw_gate=dw, act="gelu")
    R.close(dw, ref["dw_gate"], "dw_gate")


def test_ids_anywhere_and_status(P):
    """Ids that do not start at 16 bytes, sorted and not; nothing of all this ran out of time."""
    g = _gen(6)
    for kind in ("uniform", "sorted"):
        ids = _ids(kind, 30001, 700, g)
        d = torch.randn(30000, 6, generator=g)
        out = torch.empty(700, 6, device="cuda")
        P.lookup_backward(d.cuda(), ids.cuda()[1:], out)
        R.close(out, R.lookup_grad_ref(d, ids[1:], 700, 1.0))
    P.rows_status()


# -- streams, graphs, refusals --------------------------------------------------------------------

@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_other_stream_and_graph(P, dt):
    """The same bits on another stream, from two streams at once, and from two captured graphs
    replayed side by side with new inputs."""
    M, D, F, O, N = 3000, 33, 90, 20, 50
    x, wg, wu, wd, dy = _ffn_inputs(M, D, F, O, True, dt, 21)
    w = [_cuda(t) for t in (wg, wu, wd)]
    g = _gen(2)
    ids = [torch.randint(0, N, (M,), generator=g).int().cuda() for _ in range(2)]
    dys = [dy.cuda(), (dy * -0.5).cuda()]
    xs = [x.cuda(), (x * 0.5).cuda()]

    def step(i, stream=None):
        o = dict(y=torch.empty(M, O, dtype=dt, device="cuda"),
                 dx=torch.empty(M, D, dtype=dt, device="cuda"), dw=torch.empty_like(w[1]),
                 dt=torch.empty(N, D, dtype=dt, device="cuda"))
        P.ffn(xs[i], *w, o["y"], stream=stream)
        P.ffn_backward(dys[i], xs[i], *w, dx=o["dx"], dw_gate=o["dw"], stream=stream)
        P.lookup_backward(o["dx"], ids[i], o["dt"], stream=stream)
        return o

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in (0, 1):
        streams[i].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(streams[i]):
            got.append(step(i))
    torch.cuda.synchronize()
    for i in (0, 1):
        for k in want[i]:
            assert torch.equal(got[i][k], want[i][k]), k
    named = step(0, streams[1])  # outputs allocated here, kernels on the named stream
    torch.cuda.synchronize()
    for k in named:
        assert torch.equal(named[k], want[0][k]), k
    graphs, outs = [], []
    for i in (0, 1):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(i))
        graphs.append(gr)
    for _ in range(3):
        for i in (0, 1):
            for t in outs[i].values():
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            for k in want[i]:
                assert torch.equal(outs[i][k], want[i][k]), k
    xs[0].copy_(xs[1])
    dys[0].copy_(dys[1])
    ids[0].copy_(ids[1])
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    for k in want[1]:
        assert torch.equal(outs[0][k], want[1][k]), k


def test_binding_refusals(P):
    f = torch.zeros
    x, w, wd, y = f(4, 8).cuda(), f(6, 8).cuda(), f(3, 6).cuda(), f(4, 3).cuda()
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        P.ffn(x, w.half(), w, wd, y)
    with pytest.raises(TypeError):
        P.ffn(x.double(), w.double(), w.double(), wd.double(), y.double())
    with pytest.raises(ValueError):
        P.ffn(x, w, w, wd, f(4, 4).cuda())
    with pytest.raises(ValueError):
        P.ffn(x, w, f(12, 8).cuda()[::2], wd, y)
    with pytest.raises(ValueError):
        P.ffn(f(8, 4).cuda().T, w, w, wd, y)
    with pytest.raises(ValueError):
        P.ffn_backward(y, x, None, w, wd, dw_gate=w.clone())
    with pytest.raises(TypeError):
        P.lookup(x, ids.long(), x.clone())
    with pytest.raises(ValueError):
        P.lookup_backward(x, ids[:3], x.clone())
    with pytest.raises(P.SplatError) as e:  # into its own input
        P.ffn(x, w, w, f(8, 6).cuda(), x)
    assert e.value.code == -1
    with pytest.raises(P.SplatError) as e:
        P.lookup(x, ids, x)
    assert e.value.code == -1
    with pytest.raises(P.SplatError) as e:  # rows that overlap one another
        P.lookup(x, ids, f(1, 8).cuda().expand(4, 8))
    assert e.value.code == -1
    with pytest.raises(P.SplatError) as e:
        P.ffn(f(4, 129).cuda(), None, f(6, 129).cuda(), wd, y)
    assert e.value.code == -2
    with pytest.raises(P.SplatError):
        P.ffn_backward(y, x, w, w, wd)
    L = P.load_library()
    host = (ctypes.c_float * 64)()
    p = ctypes.addressof(host)
    assert L.splat_lookup(p, 8, 4, 8, ids.data_ptr(), 4, ctypes.c_float(1), 0, y.data_ptr(), 8,
                          None) == -1  # host memory
    torch.cuda.synchronize()


# -- the operators together -----------------------------------------------------------------------

@pytest.mark.parametrize("dt", DTYPES, ids=str)
def test_decode_render_and_back(P, dt):
    """Anchor rows -> Gaussians' attributes -> maps, and the way back from a map gradient, against
    the same steps in 64 bits around the render's own kernels."""
    from gaussian_splatting_raster_b200 import runner
    from synth import scenes
    sc = scenes.tiny_scene(31, 480, 40, 56, V=2, deg=1)
    ds = runner.to_device(sc)
    ws = runner.workspace_for(ds)
    out = runner.alloc_outputs(ds)
    obs = torch.rand((sc.V, sc.H, sc.W, 3), generator=_gen(1)).cuda()
    runner.render_and_score(ws, ds, obs, out)
    N, D, F, C, scale = 30, 20, 48, 5, 4.0
    g = _gen(8)
    table = torch.randn(N, D, generator=g).to(dt)
    ids = torch.arange(sc.G).div(16, rounding_mode="floor").int()
    _, wg, wu, wd, _ = _ffn_inputs(1, D, F, C, True, dt, 5)
    block = runner.FeedForward(*[_cuda(t) for t in (wg, wu, wd)], act="gelu")
    maps = torch.empty((sc.V, sc.H, sc.W, C), device="cuda")
    d = runner.decode_and_render(ws, table.cuda(), ids.cuda(), scale, block, maps)
    rows, bound = R.lookup_ref(table, ids, scale)
    R.close(d.rows, (rows, bound))
    R.close(d.feats, R.ffn_ref(d.rows.cpu(), wg, wu, wd, "gelu")["y"])
    again = torch.empty_like(maps)
    ws.render_features(d.feats.float(), again)
    assert torch.equal(maps, again)
    dmaps = torch.randn(maps.shape, generator=g).cuda()
    dtable, dblock = torch.empty_like(table.cuda()), block.zeros_like()
    runner.decode_backward(ws, ids.cuda(), scale, block, d, dmaps, dtable, dblock)
    df = torch.empty((sc.G, C), device="cuda")
    ws.scatter(dmaps, df)
    ref = R.ffn_ref(d.rows.cpu(), wg, wu, wd, "gelu", df.to(dt).cpu())
    # the scatter adds with fp64 atomics: its fp32 result may differ by a rounding between calls
    for got, name in ((dblock.w_gate, "dw_gate"), (dblock.w_up, "dw_up"),
                      (dblock.w_down, "dw_down")):
        v, b = ref[name]
        R.close(got, (v, b + (2 * R.U[dt] + 2e-7) * v.abs().max()), name)
    dx, bx = ref["dx"]
    want = torch.zeros(N, D, dtype=torch.float64).index_add_(0, ids.long(), dx) * scale
    slack = torch.zeros(N, D, dtype=torch.float64).index_add_(
        0, ids.long(), bx + (2 * R.U[dt] + 2e-7) * dx.abs().max()) * scale
    R.close(dtable, (want, slack + R.U[dt] * want.abs() + 17 * R.U32 * slack + 17 * R.U32 * (
        torch.zeros(N, D, dtype=torch.float64).index_add_(0, ids.long(), dx.abs()) * scale)))
    # and the tokens of the same step through their projection
    T = out.tokens.shape[1]
    x, _, wu, wd, _ = _ffn_inputs(1, T, 40, 12, False, dt, 6)
    feats = torch.empty((sc.G, 12), dtype=dt, device="cuda")
    runner.token_features(out, runner.FeedForward(None, wu.cuda(), wd.cuda()), feats)
    R.close(feats, R.ffn_ref(out.tokens.to(dt).cpu(), None, wu, wd, "gelu")["y"])
    ws.close()


def test_token_features_stream(P):
    """Everything of the call runs on the given stream: the current one is busy meanwhile."""
    from types import SimpleNamespace
    from gaussian_splatting_raster_b200 import runner
    dt = torch.bfloat16
    x, _, wu, wd, _ = _ffn_inputs(700, 21, 40, 12, False, dt, 7)
    out = SimpleNamespace(tokens=x.float().cuda())
    block = runner.FeedForward(None, wu.cuda(), wd.cuda())
    feats = torch.empty((700, 12), dtype=dt, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    runner.token_features(out, block, feats, stream=s)
    s.synchronize()
    with torch.cuda.stream(s):
        got = feats.cpu()
    torch.cuda.synchronize()
    R.close(got, R.ffn_ref(x, None, wu, wd, "gelu")["y"])
    P.rows_status(s)


def test_sizes_beyond_32_bits(P):
    """Sizes the library's 32-bit arguments cannot hold are refused, not cut off."""
    n = 2**32 + 1
    x, w, y = (torch.zeros(1, 1, device="cuda") for _ in range(3))
    with pytest.raises(ValueError, match="more than"):
        P.ffn(x.expand(n, 1), None, w, w, y.expand(n, 1))
    with pytest.raises(ValueError, match="more than"):
        P.lookup(x, torch.zeros(1, dtype=torch.int32, device="cuda").expand(n), y.expand(n, 1))
    with pytest.raises(ValueError, match="more than"):
        P.lookup(x.expand(n, 1), torch.zeros(1, dtype=torch.int32, device="cuda"), y)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=str)
def test_narrow_blocks_round_once(P, dt):
    """Blocks of few inputs hold hidden values in twice the bits: their outputs are rounded once."""
    M, D, F, O = 20000, 2, 104, 21
    x, wg, wu, wd, _ = _ffn_inputs(M, D, F, O, True, dt, 8)
    y = torch.empty((M, O), dtype=dt, device="cuda")
    P.ffn(x.cuda(), wg.cuda(), wu.cuda(), wd.cuda(), y, act="gelu")
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    want = (R.act(x @ wg.T, "gelu")[0] * (x @ wu.T)) @ wd.T
    # hidden values off by 2 u^2 of their size and by fp32 roundings of their arguments and of the sum
    mag = (1.13 * (x.abs() @ wg.abs().T) * (x.abs() @ wu.abs().T)) @ wd.abs().T
    e = (4 * R.U[dt] ** 2 + (F + 64) * R.ACC) * mag + F * R.TINY[dt]
    R.close(y, (want, R._held(want, e, dt)))
