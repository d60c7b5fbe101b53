"""Per-row operators called from several host threads at once."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    import gaussian_splatting_raster_b200 as P
    P.build()
    P.load_library()
    return P


def _calls(P, i, dt):
    """One thread's operators and their outputs: kernels shared with the other threads, in sizes that
    take other amounts of shared memory."""
    g = torch.Generator().manual_seed(i)
    D, F, O, M = 8 + 30 * i, 96 + 160 * i, 10 + 18 * i, 300
    x, dy = (torch.randn(M, c, generator=g).to(dt).cuda() for c in (D, O))
    wg, wu = (torch.randn(F, D, generator=g).div(D ** 0.5).to(dt).cuda() for _ in range(2))
    wd = torch.randn(O, F, generator=g).div(F ** 0.5).to(dt).cuda()
    N, n = 40 * 20 ** i, 5000
    ids = torch.randint(0, N, (n,), generator=g).int().cuda()
    d = torch.randn(n, 12, generator=g).to(dt).cuda()
    out = dict(y=torch.empty(M, O), dx=torch.empty(M, D), dwg=torch.empty(F, D),
               dwu=torch.empty(F, D), dwd=torch.empty(O, F), dt=torch.empty(N, 12))
    out = {k: v.to(dt).cuda() for k, v in out.items()}

    def run():
        P.ffn(x, wg, wu, wd, out["y"])
        P.ffn_backward(dy, x, wg, wu, wd, dx=out["dx"], dw_gate=out["dwg"], dw_up=out["dwu"],
                       dw_down=out["dwd"])
        P.lookup_backward(d, ids, out["dt"])

    return run, out


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_threads_with_other_sizes(P, dt):
    """Four threads, each on a stream of its own: no call is refused, and results are the same bits
    as alone."""
    jobs = [_calls(P, i, dt) for i in range(4)]
    want = []
    for run, out in jobs:
        run()
        want.append({k: v.clone() for k, v in out.items()})
    torch.cuda.synchronize()
    failures = []
    start = threading.Barrier(len(jobs))

    def work(i):
        run, out = jobs[i]
        try:
            stream = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(400):
                    run()
            stream.synchronize()
            for k, v in out.items():
                if not torch.equal(v, want[i][k]):
                    failures.append((i, k))
        except Exception as e:  # noqa: BLE001
            failures.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[:4]
    P.rows_status()
