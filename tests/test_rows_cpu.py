"""Per-row operators without a device: the refusals the header documents as taken before any work,
the scratch sizes, and the binding's checks."""
import ctypes

import pytest
import torch

import gaussian_splatting_raster_b200 as P
import rows_util as R

INVALID, CAPACITY, OK = -1, -2, 0
A = 1 << 20  # addresses that are never dereferenced: every call returns before it would be


@pytest.fixture(scope="module")
def L():
    P.build()
    return P.load_library()


def test_lookup_refusals(L):
    def call(table=A, ldt=8, N=4, C=8, ids=2 * A, M=4, dtype=0, out=3 * A, ldo=8):
        return L.splat_lookup(table, ldt, N, C, ids, M, ctypes.c_float(1.0), dtype, out, ldo, None)
    assert call(dtype=3) == INVALID and call(dtype=-1) == INVALID
    assert call(N=-1) == INVALID and call(M=-1) == INVALID and call(C=0) == INVALID
    assert call(C=8193) == CAPACITY
    assert call(table=None) == INVALID and call(ids=None) == INVALID and call(out=None) == INVALID
    assert call(table=A + 2) == INVALID and call(ids=2 * A + 1) == INVALID
    assert call(out=3 * A + 2) == INVALID and call(dtype=1, out=3 * A + 1) == INVALID
    assert call(ldo=7) == INVALID          # output rows that overlap
    assert call(ldt=-1) == INVALID and call(ldt=(1 << 28) + 1) == INVALID
    assert call(out=A + 64) == INVALID     # shares rows with the table
    assert call(out=2 * A) == INVALID      # shares the ids
    assert call(M=0, ids=None, out=None) == OK


def test_lookup_backward_refusals(L):
    need = L.splat_lookup_scratch(4, 4, 8)
    assert need > 0

    def call(dout=A, ldd=8, ids=2 * A, M=4, C=8, dtype=0, dt=3 * A, ldt=8, N=4, scr=4 * A,
             n=need):
        return L.splat_lookup_backward(dout, ldd, ids, M, C, ctypes.c_float(1.0), dtype, dt, ldt,
                                       N, scr, n, None)
    assert call(dtype=7) == INVALID and call(M=-1) == INVALID and call(N=-1) == INVALID
    assert call(C=0) == INVALID and call(C=8193) == CAPACITY
    assert call(n=need - 1) == INVALID and call(scr=None) == INVALID
    assert call(scr=4 * A + 8) == INVALID
    assert call(dout=None) == INVALID and call(ids=None) == INVALID and call(dt=None) == INVALID
    assert call(ldt=7) == INVALID and call(ldd=-1) == INVALID
    assert call(dt=A) == INVALID and call(scr=3 * A) == INVALID and call(scr=A) == INVALID
    assert call(N=0, dt=None) == OK


def test_ffn_refusals(L):
    def call(x=A, ldx=8, wg=2 * A, wu=3 * A, wd=4 * A, y=5 * A, ldy=8, M=4, D=8, F=8, O=8,
             dtype=0, act=0, scr=6 * A, n=1 << 16):
        return L.splat_ffn(x, ldx, wg, wu, wd, y, ldy, M, D, F, O, dtype, act, scr, n, None)
    assert call(dtype=3) == INVALID and call(act=2) == INVALID and call(act=-1) == INVALID
    for k in ("D", "F", "O"):
        assert call(**{k: 0}) == INVALID
    assert call(M=-1) == INVALID
    assert call(D=129) == CAPACITY and call(O=129) == CAPACITY and call(F=1025) == CAPACITY
    for k in ("x", "wu", "wd", "y"):
        assert call(**{k: None}) == INVALID
    assert call(y=A) == INVALID and call(y=3 * A) == INVALID
    assert call(ldy=7) == INVALID
    assert call(M=0, x=None, y=None) == OK
    for M in (1, 100, 5000):
        need = L.splat_ffn_scratch(M, 8, 8, 8, 1, 1, 0)
        if need:
            assert call(M=M, dtype=1, n=need - 1) == INVALID


def test_ffn_backward_refusals(L):
    need = L.splat_ffn_scratch(4, 8, 8, 8, 0, 1, 1)
    assert need > 0

    def call(dy=A, ldy=8, x=2 * A, ldx=8, wg=3 * A, wu=4 * A, wd=5 * A, dx=6 * A, lddx=8,
             dwg=7 * A, dwu=8 * A, dwd=9 * A, M=4, D=8, F=8, O=8, dtype=0, act=0, scr=10 * A,
             n=need):
        return L.splat_ffn_backward(dy, ldy, x, ldx, wg, wu, wd, dx, lddx, dwg, dwu, dwd, M, D, F,
                                    O, dtype, act, scr, n, None)
    assert call(dtype=3) == INVALID and call(act=2) == INVALID and call(M=-1) == INVALID
    assert call(D=129) == CAPACITY and call(O=129) == CAPACITY and call(F=1025) == CAPACITY
    assert call(n=need - 1) == INVALID and call(scr=None) == INVALID
    assert call(scr=10 * A + 8) == INVALID
    for k in ("dy", "x", "wu", "wd"):
        assert call(**{k: None}) == INVALID
    assert call(wg=None) == INVALID                                    # dwg without a gate
    assert call(dx=None, dwg=None, dwu=None, dwd=None) == INVALID      # nothing asked for
    assert call(dx=A) == INVALID and call(dwd=7 * A) == INVALID and call(lddx=7) == INVALID


def test_scratch_sizes(L):
    """Zero where there is nothing to do; monotone in the rows; 64-bit for large problems."""
    assert L.splat_lookup_scratch(0, 4, 8) == 0 and L.splat_lookup_scratch(4, 0, 8) == 0
    last = 0
    for M in (1, 100, 10_000, 1_000_000, 100_000_000):
        n = L.splat_lookup_scratch(M, 5000, 64)
        assert n >= max(last, 8 * M)
        last = n
    assert L.splat_lookup_scratch(2**31 - 1, 2**31 - 1, 64) > 2**34
    for dt in (0, 1, 2):
        assert L.splat_ffn_scratch(100, 129, 8, 8, dt, 1, 1) == 0
        assert L.splat_ffn_scratch(2**31 - 1, 128, 1024, 128, dt, 1, 1) > 0


def test_binding_checks_tensors():
    x, w = torch.zeros(4, 8), torch.zeros(8, 8)
    with pytest.raises(TypeError, match="CUDA"):
        P.ffn(x, None, w, w, x)
    with pytest.raises(TypeError, match="CUDA"):
        P.lookup(x, torch.zeros(4, dtype=torch.int32), x)
    with pytest.raises(TypeError, match="CUDA"):
        P.lookup_backward(x, torch.zeros(4, dtype=torch.int32), x)
    with pytest.raises(ValueError, match="act"):
        P.ffn(x, None, w, w, x, act="relu")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False])
def test_reference_gradients_equal_differences(kind, gated):
    """The reference formulas the kernels are held to, against central differences of <dy, y>."""
    g = torch.Generator().manual_seed(5)
    def r(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)
    t = {"x": r(5, 4), "wg": r(6, 4) if gated else None, "wu": r(6, 4), "wd": r(3, 6)}
    dy = r(5, 3)
    R.U[torch.float64] = R.TINY[torch.float64] = 0.0
    ref = R.ffn_ref(t["x"], t["wg"], t["wu"], t["wd"], kind, dy)
    names = {"x": "dx", "wg": "dw_gate", "wu": "dw_up", "wd": "dw_down"}
    for k, v in t.items():
        if v is None:
            continue
        d = r(*v.shape)
        eps = 1e-5
        L = [(dy * R.ffn_ref(*[a + s * eps * d if n == k else a for n, a in t.items()],
                             kind)["y"][0]).sum() for s in (1, -1)]
        # third derivatives of order 10 at most: eps^2 * 10 = 1e-9 of the value, 1e-11 of rounding
        assert abs((L[0] - L[1]) / (2 * eps) - (ref[names[k]][0] * d).sum()) < 1e-6
