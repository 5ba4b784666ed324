"""skgemm_i8 against exact integer sums, and its refusals.

The integer sum is exact. Its conversion to FP32 and the two products round
once each: 3 * 2^-24 relative, and bf16 adds one rounding of 2^-8. With scales
of 1 and sums below 2^24 a float output holds the sums themselves.
"""

import numpy as np
import pytest

import split_reduction_amd as sk
from oracle import ops as O
from tests.gpu_util import DEV, log, torch


def codes(rows, cols, seed, lo=-127, hi=127):
    return np.random.default_rng(seed).integers(lo, hi + 1, (rows, cols), dtype=np.int64).astype(np.int8)


def put(a, pad=0):
    """On the GPU, rows `pad` bytes longer than used and filled with 99."""
    t = torch()
    d = t.full((a.shape[0], a.shape[1] + pad), 99, dtype=t.int8, device=DEV)
    d[:, : a.shape[1]] = t.from_numpy(a).to(DEV)
    return d[:, : a.shape[1]]


def run(w, ws, x, xs, kind="bf16", pad=0, wpad=0, xpad=0, stream=None):
    t = torch()
    T, N, K = x.shape[0], w.shape[0], x.shape[1]
    C = t.full((T + 1, N + pad), -7.0, dtype=t.float32 if kind == "f32" else t.bfloat16, device=DEV)
    dev = [put(w, wpad), t.from_numpy(ws).to(DEV), put(x, xpad), t.from_numpy(xs).to(DEV)]
    t.cuda.synchronize()
    sk.skgemm_i8(dev[0], dev[1], dev[2], dev[3], C[:T, :N], T, N, K, stream=stream)
    t.cuda.synchronize()
    out = C.float().cpu().numpy()
    assert np.all(out[T] == -7) and np.all(out[:, N:] == -7), "written past the output"
    return out[:T, :N].astype(np.float64)


def scales(n, seed):
    return np.exp(np.random.default_rng(seed).uniform(-8, 2, n)).astype(np.float32)


def check(got, want, kind):
    tol = 3 * O.EPS_F32 + (O.EPS_BF16 if kind == "bf16" else 0)
    worst = np.max(np.abs(got - want) - np.abs(want) * tol, initial=-1)
    assert worst <= 0, worst


# one token to several tiles, N below, at and past a tile, K from one block to long
SIZES = [(1, 16, 16), (1, 1, 16), (1, 2048, 7168), (3, 17, 48), (16, 64, 1024), (17, 130, 272), (31, 4100, 320),
         (32, 1000, 2064), (33, 256, 128), (64, 257, 144), (65, 128, 4096), (100, 511, 1040), (128, 128, 16384),
         (129, 129, 256), (200, 1030, 528), (256, 256, 512), (300, 640, 7168), (509, 260, 1168), (513, 769, 112),
         (1000, 2048, 64), (1024, 1024, 1024), (2100, 300, 96), (4, 70000, 32), (5, 24, 131056), (70, 24, 131056)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", SIZES)
def test_i8(T, N, K):
    w, x = codes(N, K, T + N), codes(T, K, T + N + 1)
    ws, xs = scales(N, 5), scales(T, 6)
    sums, want = O.i8_ref(x, xs, w, ws)
    log(f"i8 T={T} N={N} K={K}")
    check(run(w, ws, x, xs, "bf16"), want, "bf16")
    check(run(w, ws, x, xs, "f32"), want, "f32")
    ones = np.ones
    assert np.array_equal(run(w, ones(N, np.float32), x, ones(T, np.float32), "f32"), sums.astype(np.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", [(1, 100, 256), (20, 300, 1024), (150, 1000, 512), (600, 515, 272), (1100, 1100, 160)])
def test_i8_strides(T, N, K):
    """Rows inside wider matrices; the bytes between them are not read as values."""
    w, x, ws, xs = codes(N, K, 1), codes(T, K, 2), scales(N, 3), scales(T, 4)
    _, want = O.i8_ref(x, xs, w, ws)
    for kind, pad in (("bf16", 3), ("f32", 1), ("bf16", 8)):
        log(f"i8 strides T={T} N={N} K={K} {kind} pad={pad}")
        check(run(w, ws, x, xs, kind, pad=pad, wpad=48, xpad=16), want, kind)


# Every tile shape, and the kernel without tiles (6), pinned: sizes below, at and
# past a tile, K that ends inside a step, and K split over workgroups, among them
# calls of more tiles than one round of workgroups, of which only the last are
# split.
@pytest.mark.gpu
@pytest.mark.parametrize("shape", range(7))
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (33, 65, 144), (256, 256, 128), (257, 300, 1040), (700, 129, 4112)])
def test_i8_shapes(T, N, K, shape, tune):
    w, x, ws, xs = codes(N, K, 1), codes(T, K, 2), scales(N, 3), scales(T, 4)
    _, want = O.i8_ref(x, xs, w, ws)
    tune("i8_shape", shape)
    got = {}
    for S in (1, 2, 3, 5, 8):
        tune("i8_split", S)
        log(f"i8 shape {shape} split {S} T={T} N={N} K={K}")
        got[S] = run(w, ws, x, xs, "f32")
        check(got[S], want, "f32")
        assert np.array_equal(got[S], got[1]), "a split changes bits"
    check(run(w, ws, x, xs, "bf16"), want, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("shape,T,N,K", [(0, 4000, 4300, 400), (1, 4000, 2300, 400), (2, 3000, 3100, 272),
                                         (3, 2000, 2200, 400), (4, 1500, 1600, 400), (5, 1000, 1700, 400)])
def test_i8_last_round_split(shape, T, N, K, tune):
    w, x, ws, xs = codes(N, K, 1), codes(T, K, 2), scales(N, 3), scales(T, 4)
    _, want = O.i8_ref(x, xs, w, ws)
    tune("i8_shape", shape)
    for S in (1, 2, 4):
        tune("i8_split", S)
        log(f"i8 last round shape {shape} split {S}")
        check(run(w, ws, x, xs, "f32"), want, "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 300])
def test_i8_extremes(T):
    """The largest sums: every code -128 (or 127 against -128) at the longest K."""
    N, K = 40, 131056
    w, x = np.full((N, K), -128, np.int8), np.full((T, K), -128, np.int8)
    x[:, 1::2] = 127
    w[::2] = 127
    one = lambda n: np.ones(n, np.float32)  # noqa: E731
    sums, _ = O.i8_ref(x, one(T), w, one(N))
    log(f"i8 extremes T={T}")
    assert np.array_equal(run(w, one(N), x, one(T), "f32"), sums.astype(np.float32))
    x[:] = -128
    w[:] = -128
    sums, _ = O.i8_ref(x, one(T), w, one(N))
    assert sums.max() < 2**31
    assert np.array_equal(run(w, one(N), x, one(T), "f32"), sums.astype(np.float32))


@pytest.mark.gpu
def test_i8_zero_k_and_nan_scale():
    t = torch()
    C = t.full((3, 20), 5.0, device=DEV)
    s = t.ones(20, device=DEV)
    sk.skgemm_i8(0, s, 0, s, C, 3, 20, 0)
    t.cuda.synchronize()
    assert not C.any()
    w, x = codes(20, 64, 1), codes(3, 64, 2)
    xs = np.array([1, np.nan, 2], np.float32)
    got = run(w, np.ones(20, np.float32), x, xs, "f32")
    assert np.isnan(got[1]).all() and np.isfinite(got[[0, 2]]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", [(1, 2048, 7168), (48, 1024, 4096), (300, 512, 2048)])
def test_i8_captured_and_streams(T, N, K):
    """Replays between eager calls of other sizes on the same stream give the
    eager bits; so do calls on two streams at once."""
    t = torch()
    w, x, ws, xs = codes(N, K, 1), codes(T, K, 2), scales(N, 3), scales(T, 4)
    W, X, WS, XS = put(w), put(x), t.from_numpy(ws).to(DEV), t.from_numpy(xs).to(DEV)
    s, s2 = t.cuda.Stream(), t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    s2.wait_stream(t.cuda.current_stream())
    C, C2 = t.empty(T, N, device=DEV), t.empty(T, N, device=DEV)
    for _ in range(4):
        sk.skgemm_i8(W, WS, X, XS, C, T, N, K, stream=s)
        sk.skgemm_i8(W, WS, X, XS, C2, T, N, K, stream=s2)
    t.cuda.synchronize()
    assert t.equal(C, C2)
    check(C.cpu().double().numpy(), O.i8_ref(x, xs, w, ws)[1], "f32")
    want = C.clone()
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr, stream=s):
        sk.skgemm_i8(W, WS, X, XS, C, T, N, K, stream=s)
    small = t.empty(1, 100, device=DEV)
    for _ in range(3):
        C.zero_()
        t.cuda.synchronize()
        with t.cuda.stream(s):
            gr.replay()
        t.cuda.synchronize()
        assert t.equal(C, want)
        sk.skgemm_i8(W, WS, X, XS, small, 1, 100, K, stream=s)
        t.cuda.synchronize()
        assert t.equal(small[0], want[0, :100])


def test_i8_refusals():
    f = sk.lib().skgemm_i8
    a = 1 << 20

    def call(W=a, ws=a, X=a, xs=a, C=a, T=2, N=32, K=64, fmt=0, wst=64, xst=64, cst=64):
        return f(W, ws, X, xs, C, T, N, K, fmt, wst, xst, cst, None)

    assert call(T=-1) == call(N=-1) == call(K=-16) == call(fmt=1) == call(fmt=2) == sk.SKGEMM_EINVAL
    assert call(K=24) == call(K=131072) == call(N=(1 << 18) + 1) == sk.SKGEMM_ESHAPE
    assert call(W=None) == call(X=None) == call(C=None) == call(ws=None) == call(xs=None) == sk.SKGEMM_EINVAL
    assert call(W=a + 8) == call(X=a + 8) == call(C=a + 8) == call(ws=a + 2) == call(xs=a + 2) == sk.SKGEMM_EALIGN
    assert call(wst=72) == call(xst=72) == call(cst=65) == call(fmt=3, cst=130) == sk.SKGEMM_EALIGN
    assert call(wst=48) == call(xst=48) == call(cst=62) == call(fmt=3, cst=124) == sk.SKGEMM_EINVAL
    assert call(wst=(1 << 22) + 16) == call(xst=(1 << 22) + 16) == sk.SKGEMM_ESHAPE
    assert call(W=None, X=None, C=None, T=0) == call(W=None, C=None, N=0) == sk.SKGEMM_OK


def test_i8_binding_refusals():
    t = torch()
    with pytest.raises(sk.SkgemmError) as e:
        sk.skgemm_i8(t.zeros(32, 64, dtype=t.int8), 1 << 20, 1 << 20, 1 << 20, 1 << 20, 2, 32, 64)
    assert e.value.code == sk.SKGEMM_EINVAL and "not on the GPU" in str(e.value)
