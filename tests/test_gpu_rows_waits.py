"""A bounded wait that runs out: the lookup gradient's sort, built with no patience at all, so that a CTA
gives up at the first count of a predecessor that is not there yet. Its results mean nothing then; it
ends, writes nothing but its outputs and scratch, and says so once. (The waits of the feed-forward
block's kernels are tested on a model only, test_rows_protocol.)"""
import ctypes
import importlib
import os
import subprocess

import pytest
import torch

import rows_util as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    B = importlib.import_module("gaussian_splatting_raster_b200.build")
    d = tmp_path_factory.mktemp("impatient")
    stub = d / "stub.cu"  # the status call asks the feed-forward block's kernels too
    stub.write_text('#include "rows.cuh"\nnamespace splat { namespace rows {\n'
                    "cudaError_t ffn_status_take(unsigned int* out, cudaStream_t) "
                    "{ *out = 0; return cudaSuccess; }\n} }\n")
    lib = d / "lib.so"
    subprocess.check_call([B.nvcc(), *B.NVCC_FLAGS, "-DSPLAT_LOOKUP_WAIT_CLOCKS=-1",
                           "-I", os.path.join(B.ROOT, "include"), "-I", B.CSRC, str(stub),
                           *[os.path.join(B.CSRC, s) for s in ("rows.cu", "lookup.cu")],
                           "-o", str(lib)])
    L = ctypes.CDLL(str(lib))
    V, I, LL, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    L.splat_lookup_scratch.argtypes, L.splat_lookup_scratch.restype = [I, I, I], LL
    L.splat_lookup_backward.argtypes = [V, LL, V, I, I, F, I, V, LL, I, V, LL, V]
    L.splat_rows_status.argtypes = [V]
    return L


@pytest.mark.parametrize("M,N", [(2000000, 70000), (2000000, 2000), (1300000, 1200000)])
def test_sort_wait_runs_out(impatient, M, N):
    """Every eighth stretch of 8,192 ids (what one CTA counts) is one id: its CTA counts them one after
    the other and is late."""
    import gaussian_splatting_raster_b200 as P
    L, C, guard = impatient, 20, 4096
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(0, N, (M,), generator=g).int()
    ids[(torch.arange(M) // 8192) % 8 == 0] = N // 2
    ids = ids.cuda()
    dout = torch.randn(M, C, generator=g).cuda()
    need = L.splat_lookup_scratch(M, N, C)
    scratch = torch.full((need + 2 * guard,), 171, dtype=torch.uint8, device="cuda")
    wide = torch.full((N * C + 2 * guard,), 7.0, device="cuda")
    codes = []
    for _ in range(10):
        rc = L.splat_lookup_backward(dout.data_ptr(), C, ids.data_ptr(), M, C, 1.0, 0,
                                     wide[guard:].data_ptr(), C, N, scratch[guard:].data_ptr(),
                                     need, None)
        assert rc == 0
        codes.append(L.splat_rows_status(None))
        assert L.splat_rows_status(None) == 0  # told once
    torch.cuda.synchronize()
    assert set(codes) <= {0, -6} and -6 in codes
    for t, v in ((scratch, 171), (wide, 7)):
        assert (t[:guard] == v).all() and (t[-guard:] == v).all()
    # the library itself, in the same process
    out = torch.empty(N, C, device="cuda")
    P.lookup_backward(dout, ids, out)
    P.rows_status()
    R.close(out, R.lookup_grad_ref(dout.cpu(), ids.cpu(), N, 1.0))
