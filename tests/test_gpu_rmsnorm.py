"""skgemm_rmsnorm against the fp64 formula, and its refusals.

Bounds, counted in roundings of half a step (2^-24 relative in FP32):
* the row's 1/rms: one rounding of h (it counts twice in h^2), at most 32
  fused additions in a thread, 6 + 15 across the workgroup, all terms
  positive, halved by the square root, and four more (mean, eps, root,
  division): below 36. With max|h g| (two roundings), the division by the
  largest code and the product, a scale is within 40 * 2^-24;
* bf16 y: the same and the products' two, below 40, and one bf16 rounding;
* a code before its rounding: h, h g, the largest h g (2), the division by it
  and the product: 6 * 2^-24 of the largest code at most; then half a code
  (int8), or half an E4M3 step (2^-4 of the value, 2^-10 below the smallest
  normal).
"""

import numpy as np
import pytest

import split_reduction_amd as sk
from oracle import formats as F
from oracle import ops as O
from tests.gpu_util import DEV, log, torch

ULP = O.EPS_F32


def rows(T, H, seed, spread=True):
    rng = np.random.default_rng(seed)
    t = torch()
    x = rng.standard_normal((T, H)).astype(np.float32)
    r = 2 * rng.standard_normal((T, H)).astype(np.float32)
    if spread:  # rows of very different sizes
        x *= np.exp(rng.uniform(-6, 6, (T, 1))).astype(np.float32)
    g = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
    return [t.from_numpy(a).to(t.bfloat16) for a in (x, r, g)]


def f64(a):
    return None if a is None else a.float().double().cpu().numpy()


def check(x, r, g, ro, y, ys, eps, fmt):
    h, want = O.rmsnorm_ref(f64(x), f64(r), f64(g), eps)
    if ro is not None:
        got = f64(ro)
        fine = np.isfinite(h)
        assert np.array_equal(np.isnan(got), np.isnan(h))
        assert np.all(np.abs(got - h)[fine] <= np.abs(h)[fine] * (O.EPS_BF16 + ULP) + 2.0**-133)
    bad = np.isnan(want).any(axis=1)
    if fmt == "bf16":
        got = f64(y)
        assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
        err = np.abs(got - want)[~bad] - 2.0**-133
        assert np.all(err <= np.abs(want)[~bad] * (O.EPS_BF16 + 40 * ULP))
        return
    scale = ys.double().cpu().numpy()
    assert np.isnan(scale[bad]).all()
    ref = O.row_scale(want[~bad], fmt)
    assert np.all(np.abs(scale[~bad] - ref) <= ref * 40 * ULP)
    code = y.cpu().view(torch().uint8).numpy()
    code = code.view(np.int8).astype(np.float64) if fmt == "i8" else F.e4m3_value(code)
    code = code[~bad]
    top = O.TOP_CODE[fmt]
    with np.errstate(invalid="ignore", divide="ignore"):
        v = np.where(ref[:, None] > 0, want[~bad] / ref[:, None], 0.0)
    half = 0.5 if fmt == "i8" else np.maximum(np.abs(v) * O.EPS_E4M3, 2.0**-10)
    off = np.abs(code - v) - half
    log(f"  {fmt}: largest distance past half a code {off.max():.3g}")
    assert np.all(off <= 6 * ULP * top * (1 + O.EPS_E4M3))


def run(x, r, g, fmt, eps=1e-6, keep=True, T=None, H=None, stream=None):
    t = torch()
    T, H = x.shape if T is None else (T, H)
    dev = [None if a is None else a.to(DEV) for a in (x, r, g)]
    ro = t.full((T, H), float("nan"), dtype=t.bfloat16, device=DEV) if keep else None
    y = t.full((T, H), 0x55, dtype=t.uint8, device=DEV) if fmt != "bf16" else t.full((T, H), 7e7, dtype=t.bfloat16, device=DEV)
    ys = t.full((T,), -1.0, device=DEV)
    sk.skgemm_rmsnorm(dev[0], dev[1], dev[2], ro, y, ys, T, H, eps, fmt, stream=stream)
    t.cuda.synchronize()
    return ro, y, ys


SIZES = [(1, 8), (1, 7168), (3, 1000), (5, 512), (2, 16384), (2, 32768), (257, 1352), (64, 8184), (700, 2048), (1500, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("T,H", SIZES)
def test_rmsnorm(T, H, fmt):
    x, r, g = rows(T, H, seed=T * 7 + H)
    log(f"rmsnorm T={T} H={H} {fmt}")
    check(x, r, g, *run(x, r, g, fmt), 1e-6, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,fmt", [(1100, 4104, "i8"), (1100, 4104, "bf16"), (9400, 4096, "e4m3"), (5000, 8192, "i8")])
def test_rmsnorm_many_rows(T, H, fmt):
    """Several vectors a thread, and inputs past the last cache."""
    x, r, g = rows(T, H, seed=T)
    log(f"rmsnorm T={T} H={H} {fmt}")
    check(x, r, g, *run(x, r, g, fmt), 1e-6, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("res,gain,keep", [(False, True, True), (True, False, False), (False, False, False)])
def test_rmsnorm_without(res, gain, keep, fmt):
    x, r, g = rows(9, 3000, seed=5)
    r, g = (r if res else None), (g if gain else None)
    check(x, r, g, *run(x, r, g, fmt, keep=keep, eps=1e-5), 1e-5, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("H", [64, 7168])
def test_rmsnorm_far_values(H, fmt):
    """Zeros, squares past FP32's range at both ends, infinities and NaN."""
    t = torch()
    x, _, g = rows(8, H, seed=11, spread=False)
    x[0] = 0
    x[1] = x[1] * 1e30
    x[2] = x[2] * 1e-30
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5, 7] = float("-inf")
    x[6] = x[6].sign() * 3.38e38
    x[7] = 0
    x[7, H - 1] = 1e-38
    log(f"rmsnorm far values H={H} {fmt}")
    ro, y, ys = run(x, None, g, fmt)
    check(x, None, g, ro, y, ys, 1e-6, fmt)
    if fmt != "bf16":
        assert ys[0].item() == 0 and not y[0].view(t.uint8).any()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("H,T", [(64, 9), (7168, 9), (7168, 1100), (16384, 3)])
@pytest.mark.parametrize("gain", [float("nan"), float("inf"), float("-inf")])
def test_rmsnorm_gain_not_finite(H, T, gain, fmt):
    """An element of G that is no number shows: in bf16 where it is, else in the
    scale. Rows whose squares pass FP32's range, and a row with a zero there."""
    t = torch()
    x, r, g = rows(T, H, seed=2, spread=False)
    at = H - 5
    g[at] = gain
    x[1], r[1] = x[1] * 1e30, 0
    x[2, at] = r[2, at] = 0  # 0 * inf is NaN
    log(f"rmsnorm gain {gain} T={T} H={H} {fmt}")
    ro, y, ys = run(x, r, g, fmt)
    nan = np.isnan(gain) | (f64(x)[:, at] + f64(r)[:, at] == 0)  # row 2, and where a sum happens to be 0
    assert nan[2]
    if fmt == "bf16":
        got = f64(y)
        _, want = O.rmsnorm_ref(f64(x), f64(r), np.where(np.arange(H) == at, 0.0, f64(g)), 1e-6)
        rest = np.arange(H) != at
        assert np.all(np.abs(got - want)[:, rest] <= np.abs(want)[:, rest] * (O.EPS_BF16 + 40 * ULP) + 2.0**-133)
        got = got[:, at]
    else:
        got = ys.double().cpu().numpy()
    assert np.isnan(got[nan]).all() and np.isinf(got[~nan]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("H", [64, 7168])
def test_rmsnorm_far_gain(H, fmt):
    """G near the type's largest value, where h G passes FP32's range and y does
    not; for codes also a y that passes it and a scale that does not."""
    t = torch()
    rng = np.random.default_rng(H)
    x = rng.uniform(0.55, 0.65, (4, H)) * rng.choice([-1, 1], (4, H))
    x *= np.array([1, 1e10, 3e38, 1e-3])[:, None]
    g = np.where(rng.random(H) < 0.5, 3e38 * rng.choice([-1, 1], H), rng.standard_normal(H))
    g[3] = 3e38
    if fmt != "bf16":
        x[:2, 3] *= 3
    x, g = (t.from_numpy(a).to(t.bfloat16) for a in (x, g))
    log(f"rmsnorm far gain H={H} {fmt}")
    check(x, None, g, *run(x, None, g, fmt), 1e-6, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["i8", "bf16"])
def test_rmsnorm_strides_in_place_and_stream(fmt):
    """Rows inside wider matrices, R_out on top of R, another stream."""
    t = torch()
    T, H = 33, 1352
    x, r, g = rows(T, H, seed=3)
    wide = lambda a, n: t.full((T, H + n), 3.0, dtype=t.bfloat16, device=DEV)  # noqa: E731
    X, R = wide(x, 24), wide(r, 8)
    X[:, :H], R[:, :H] = x.to(DEV), r.to(DEV)
    kind = t.uint8 if fmt == "i8" else t.bfloat16
    Y = t.full((T, H + 40), 9, dtype=kind, device=DEV)
    ys = t.empty(T, device=DEV)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    sk.skgemm_rmsnorm(X[:, :H], R[:, :H], g.to(DEV), R[:, :H], Y[:, :H], ys, T, H, 1e-6, fmt, stream=s)
    t.cuda.synchronize()
    check(x, r, g, R[:, :H].contiguous(), Y[:, :H].contiguous(), ys, 1e-6, fmt)
    assert (X[:, H:] == 3).all() and (R[:, H:] == 3).all() and (Y[:, H:] == 9).all()


@pytest.mark.gpu
def test_rmsnorm_captured():
    t = torch()
    x, r, g = (a.to(DEV) for a in rows(17, 2048, seed=8))
    y, ys = t.empty(17, 2048, dtype=t.int8, device=DEV), t.empty(17, device=DEV)
    ro = t.empty_like(x)
    sk.skgemm_rmsnorm(x, r, g, ro, y, ys, 17, 2048, 1e-6, "i8")
    t.cuda.synchronize()
    want = [a.clone() for a in (ro, y, ys)]
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr):
        sk.skgemm_rmsnorm(x, r, g, ro, y, ys, 17, 2048, 1e-6, "i8")
    for _ in range(3):
        for a in (ro, y, ys):
            a.zero_()
        gr.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip((ro, y, ys), want))


def test_rmsnorm_refusals():
    """Every refusal comes before any device work: the addresses are made up."""
    f = sk.lib().skgemm_rmsnorm
    a = 1 << 20

    def call(X=a, R=a, G=a, RO=a, Y=a, S=a, T=2, H=64, eps=1e-6, fmt=1, xs=128, rs=128, ros=128, ys=64):
        return f(X, R, G, RO, Y, S, T, H, eps, fmt, xs, rs, ros, ys, None)

    assert call(T=-1) == call(H=-8) == call(fmt=3) == call(fmt=-1) == sk.SKGEMM_EINVAL
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        assert call(eps=eps) == sk.SKGEMM_EINVAL
    assert call(H=60) == call(H=32776) == sk.SKGEMM_ESHAPE
    assert call(X=None) == call(Y=None) == call(S=None) == sk.SKGEMM_EINVAL
    for name in ("X", "R", "G", "RO", "Y"):
        assert call(**{name: a + 8}) == sk.SKGEMM_EALIGN
    assert call(S=a + 2) == sk.SKGEMM_EALIGN
    assert call(xs=136) == call(rs=136) == call(ros=136) == call(ys=68) == sk.SKGEMM_EALIGN
    assert call(ys=56) == call(ros=112) == call(fmt=0, ys=112) == sk.SKGEMM_EINVAL
    assert call(X=None, T=0) == call(X=None, H=0) == sk.SKGEMM_OK


def test_rmsnorm_binding_refusals():
    t = torch()
    x = t.zeros(4, 64, dtype=t.bfloat16)
    for bad in (x, t.zeros(4, 64)):
        with pytest.raises(sk.SkgemmError) as e:
            sk.skgemm_rmsnorm(bad, None, None, None, 1 << 20, 1 << 20, 4, 64, 1e-6, "i8")
        assert e.value.code == sk.SKGEMM_EINVAL
    with pytest.raises(sk.SkgemmError) as e:
        sk.skgemm_rmsnorm(1 << 20, None, None, None, 1 << 20, 1 << 20, 4, 64, 1e-6, "int4")
    assert e.value.code == sk.SKGEMM_EINVAL
