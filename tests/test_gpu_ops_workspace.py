"""The workspace of the operators around the layers: what a capture needs, what
skgemm_release frees, and calls of both kinds that use it in turn on one stream."""

import numpy as np
import pytest

import split_reduction_amd as sk
from oracle import ops as O
from tests.gpu_util import DEV, torch


def call(Z, out, T, V, k, stream):
    sk.skgemm_logprobs(Z, None, None, out[0], out[1], out[2], out[3], T, V, k, stream=stream)


@pytest.mark.gpu
def test_capture_needs_the_workspace():
    t = torch()
    T, V, k = 1, 100000, 4
    Z = t.randn(T, V, device=DEV)
    out = [t.zeros(T, device=DEV), t.zeros(T, device=DEV), t.zeros(T, k, device=DEV), t.zeros(T, k, dtype=t.int64, device=DEV)]
    t.cuda.synchronize()
    sk.skgemm_release()  # no stream has a workspace now
    s = t.cuda.Stream()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        out[0].zero_()
        with pytest.raises(sk.SkgemmError) as e:
            call(Z, out, T, V, k, s)
    assert e.value.code == sk.SKGEMM_ENOMEM
    sk.skgemm_reserve_ops(s)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        call(Z, out, T, V, k, s)
    for _ in range(3):
        for a in out:
            a.zero_()
        t.cuda.synchronize()
        with t.cuda.stream(s):
            g.replay()
        t.cuda.synchronize()
        assert t.equal(out[3][0], t.topk(Z[0], k).indices)
    del g


@pytest.mark.gpu
def test_operators_in_turn_on_one_workspace():
    """Split products and split rows leave the counters at zero for each other."""
    t = torch()
    rng = np.random.default_rng(1)
    w, x = (rng.integers(-127, 128, s).astype(np.int8) for s in ((500, 8192), (40, 8192)))
    one = lambda n: np.ones(n, np.float32)  # noqa: E731
    sums, _ = O.i8_ref(x, one(40), w, one(500))
    W, X = t.from_numpy(w).to(DEV), t.from_numpy(x).to(DEV)
    ws, xs, C = t.ones(500, device=DEV), t.ones(40, device=DEV), t.empty(40, 500, device=DEV)
    Z = t.randn(7, 60001, device=DEV)
    out = [t.empty(7, device=DEV), t.empty(7, device=DEV), t.empty(7, 9, device=DEV), t.empty(7, 9, dtype=t.int64, device=DEV)]
    want = t.topk(Z, 9).indices
    for _ in range(5):
        C.zero_()
        out[3].zero_()
        sk.skgemm_i8(W, ws, X, xs, C, 40, 500, 8192)
        call(Z, out, 7, 60001, 9, None)
        t.cuda.synchronize()
        assert np.array_equal(C.cpu().numpy(), sums.astype(np.float32))
        assert t.equal(out[3], want)
    t.cuda.synchronize()
    sk.skgemm_release()
    sk.skgemm_i8(W, ws, X, xs, C, 40, 500, 8192)  # allocated again
    t.cuda.synchronize()
    assert np.array_equal(C.cpu().numpy(), sums.astype(np.float32))


def test_negative_stride_refused():
    for f in (lambda: sk.skgemm_rmsnorm(1 << 20, None, None, None, 1 << 20, None, 4, 64, 1e-6, "bf16", x_stride=-128),
              lambda: sk.skgemm_logprobs(1 << 20, None, None, None, None, None, None, 4, 64, stride=-128)):
        with pytest.raises(sk.SkgemmError) as e:
            f()
        assert e.value.code == sk.SKGEMM_EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("reserve", [sk.skgemm_reserve_ops, lambda s: sk.skgemm_reserve(64, 4096, 4, s)])
def test_reserve_has_cleared_the_workspace(reserve):
    """A reserve on a busy stream returns with the workspace's counters cleared:
    what is captured there may be replayed on a stream that waits for nothing."""
    t = torch()
    sk.skgemm_release()
    s = t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.stream(s):
        t.cuda._sleep(100_000_000)  # tens of milliseconds
    assert not s.query()
    reserve(s)
    assert s.query()
    sk.skgemm_release()


@pytest.mark.gpu
def test_replay_on_another_stream():
    t = torch()
    T, V, k = 1, 100000, 4
    Z = t.randn(T, V, device=DEV)
    out = [t.zeros(T, device=DEV), t.zeros(T, device=DEV), t.zeros(T, k, device=DEV), t.zeros(T, k, dtype=t.int64, device=DEV)]
    sk.skgemm_release()
    s, s2 = t.cuda.Stream(), t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.stream(s):
        t.cuda._sleep(50_000_000)
    sk.skgemm_reserve_ops(s)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        call(Z, out, T, V, k, s)
    with t.cuda.stream(s2):
        for _ in range(3):
            g.replay()
    t.cuda.synchronize()
    assert t.equal(out[3][0], t.topk(Z[0], k).indices)
    del g
    sk.skgemm_release()
