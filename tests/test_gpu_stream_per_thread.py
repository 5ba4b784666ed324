"""hipStreamPerThread: one handle, a stream and a workspace of each host thread."""

import threading

import numpy as np
import pytest

import split_reduction_amd as sk
from oracle import ops as O
from tests.gpu_util import DEV, torch

PER_THREAD = 2  # hipStreamPerThread


def in_threads(n, f):
    """f(i) in n threads at once; the first error of any is raised here."""
    errors = []

    def run(i):
        try:
            torch().cuda.set_device(0)
            f(i)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    if errors:
        raise errors[0]


@pytest.mark.gpu
@pytest.mark.parametrize("reserve,size", [(lambda: sk.skgemm_reserve_ops(PER_THREAD), 65 << 20),
                                          (lambda: sk.skgemm_reserve(128, 65536, 8, PER_THREAD), 256 << 20)])
def test_each_thread_has_its_workspace(reserve, size):
    t = torch()
    sk.skgemm_release()
    free = []

    def note(_):
        reserve()
        reserve()  # the thread's own: nothing new
        t.cuda.synchronize()
        free.append(t.cuda.mem_get_info()[0])

    t.cuda.synchronize()
    free.append(t.cuda.mem_get_info()[0])
    for _ in range(3):
        in_threads(1, note)
    steps = [a - b for a, b in zip(free[1:], free[2:])]  # the first thread's holds the kernels' code too
    sk.skgemm_release()
    assert all(size <= s < 2 * size for s in steps), steps


@pytest.mark.gpu
def test_threads_at_once():
    t = torch()
    sk.skgemm_release()
    rng = np.random.default_rng(0)
    N, K, T, V, k, n = 500, 8192, 40, 131072, 9, 3
    one = np.ones
    w = rng.integers(-127, 128, (N, K)).astype(np.int8)
    W, ws, xs = t.from_numpy(w).to(DEV), t.ones(N, device=DEV), t.ones(T, device=DEV)
    x = [rng.integers(-127, 128, (T, K)).astype(np.int8) for _ in range(n)]
    X = [t.from_numpy(a).to(DEV) for a in x]
    Z = [t.randn(2, V, device=DEV) for _ in range(n)]
    C = [t.zeros(40, T, N, device=DEV) for _ in range(n)]
    ids = [t.zeros(40, 2, k, dtype=t.int64, device=DEV) for _ in range(n)]
    top = [t.zeros(2, k, device=DEV) for _ in range(n)]
    t.cuda.synchronize()

    def work(i):
        for j in range(40):
            sk.skgemm_i8(W, ws, X[i], xs, C[i][j], T, N, K, stream=PER_THREAD)
            sk.skgemm_logprobs(Z[i], None, None, None, None, top[i], ids[i][j], 2, V, k, stream=PER_THREAD)

    in_threads(n, work)
    t.cuda.synchronize()
    for i in range(n):
        want = O.i8_ref(x[i], one(T), w, one(N))[0].astype(np.float32)
        got = C[i].cpu().numpy()
        assert all(np.array_equal(a, want) for a in got), i
        best = t.topk(Z[i], k).indices
        assert all(t.equal(a, best) for a in ids[i]), i
    sk.skgemm_release()
