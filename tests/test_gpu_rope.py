"""skgemm_rope and skgemm_rope_append against the fp64 formula, and their refusals.

Bounds, counted in roundings of half a step (2^-24 relative in FP32):
* 1/rms of a head: 16 fused additions in a lane and 4 across lanes, halved by the
  root, then mean, eps, root and division: below 20; with the two products 22;
* a cosine or sine: 2 of its own, and the angle's rounding to part of a turn, 2^-25
  turns = 0.2 * 2^-20 radians = 3.2 * 2^-24 of the pair's size; amplitude 1; the two
  products and their sum 3. Together a pair's size |a| + |b| times 32 * 2^-24;
* bf16: one rounding more; E4M3: the value's division by the scale (2), then half a
  step of the code (2^-4 of it, 2^-10 below the smallest normal).
Positions stay below 2^22, where fp64's own product is off by less than 2^-30.
"""

import numpy as np
import pytest

import split_reduction_amd as sk
from oracle import formats as F
from oracle import ops as O
from tests.gpu_util import DEV, log, torch

ULP = O.EPS_F32
FREQ = lambda rot, base=10000.0: (base ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)  # noqa: E731


def f64(a):
    return None if a is None else a.float().double().cpu().numpy()


def bf16(a):
    t = torch()
    return t.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(t.bfloat16)


def heads(T, H, D, seed, spread=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, D))
    if spread:
        x *= np.exp(rng.uniform(-4, 4, (T, H, 1)))
    return bf16(x), bf16(1 + 0.2 * rng.standard_normal(D)), rng


def close(got, ref, size, what):
    err = np.abs(got - ref) - O.EPS_BF16 * np.abs(ref)
    tol = size * 32 * ULP * (1 + O.EPS_BF16) + 2.0**-133
    assert np.isfinite(got).all() and np.all(err <= tol), (what, (err / np.maximum(tol, 1e-300)).max())


def close_codes(code, ref, size, scale, what):
    got, want = F.e4m3_value(code), np.clip(ref / scale, -448, 448)
    half = np.maximum(np.abs(want) * O.EPS_E4M3, 2.0**-10)
    tol = (34 * ULP * size / scale) * (1 + O.EPS_E4M3)
    assert np.all(np.abs(got - want) <= half + tol), what


CASES = [  # T, H, D, rot, layout
    (1, 1, 64, 64, "half"), (1, 16, 128, 128, "half"), (3, 5, 128, 64, "interleaved"), (2, 80, 128, 128, "half"),
    (67, 7, 256, 256, "half"), (130, 3, 16, 16, "interleaved"), (33, 2, 80, 32, "half"), (9, 33, 96, 96, "interleaved"),
    (5, 17, 192, 48, "half"), (1500, 1, 128, 128, "half"), (1100, 40, 64, 16, "interleaved"), (257, 12, 240, 0, "half"),
    (2, 300, 32, 32, "half"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,H,D,rot,layout", CASES)
def test_rope(T, H, D, rot, layout, norm):
    t = torch()
    x, g, rng = heads(T, H, D, T + H + D)
    pos, freq = rng.integers(0, 1 << 22, T), FREQ(rot)
    log(f"rope T={T} H={H} D={D} rot={rot} {layout} norm={norm}")
    ref, size = O.rope_ref(f64(x), f64(g) if norm else None, freq, pos, rot, layout, 1e-5, 1.25)
    y = t.full((T, H, D), 7e7, dtype=t.bfloat16, device=DEV)
    args = (t.from_numpy(freq).to(DEV) if rot else None, t.from_numpy(pos).to(DEV) if rot else None)
    sk.skgemm_rope(x.to(DEV), g.to(DEV) if norm else None, *args, y, T, H, D, rot, layout, 1e-5, 1.25)
    t.cuda.synchronize()
    close(f64(y), ref, size, "rope")


@pytest.mark.gpu
def test_rope_positions_and_scaled_frequencies():
    """Positions 0, 1, far and negative; frequencies of a context stretched fourfold."""
    t = torch()
    T, H, D = 6, 4, 128
    x, _, _ = heads(T, H, D, 4)
    pos = np.array([0, 1, -1, 4096, (1 << 22) - 1, 131071])
    freq = FREQ(D)
    ramp = np.clip((np.arange(D // 2) - 20) / 20, 0, 1)
    freq = (freq * (1 - ramp) + freq / 4 * ramp).astype(np.float32)
    ref, size = O.rope_ref(f64(x), None, freq, pos, D, "half", amplitude=1.1386)
    y = t.empty(T, H * D, dtype=t.bfloat16, device=DEV)
    sk.skgemm_rope(x.to(DEV), None, t.from_numpy(freq).to(DEV), t.from_numpy(pos).to(DEV), y, T, H, D, D, amplitude=1.1386)
    t.cuda.synchronize()
    close(f64(y).reshape(T, H, D), ref, size, "scaled")
    assert t.equal(y[0].cpu().float(), (x[0].float() * np.float32(1.1386)).to(t.bfloat16).flatten().float())


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_far_values(layout):
    """Zeros, squares past FP32's range at both ends, infinities and NaN, each head for itself."""
    t = torch()
    T, H, D = 2, 8, 128
    x, g, _ = heads(T, H, D, 9, spread=False)
    x[:, 0] = 0
    x[:, 1] *= 1e30
    x[:, 2] *= 1e-30
    x[:, 3, 5] = float("inf")
    x[:, 4, 100] = float("nan")
    x[:, 5] = x[:, 5].sign() * 3.38e38
    x[:, 6, 1:] = 0
    pos, freq = np.array([3, 70000]), FREQ(64)
    ok = [0, 1, 2, 5, 6, 7]
    ref, size = O.rope_ref(f64(x)[:, ok], f64(g), freq, pos, 64, layout)
    y = t.empty(T, H, D, dtype=t.bfloat16, device=DEV)
    sk.skgemm_rope(x.to(DEV), g.to(DEV), t.from_numpy(freq).to(DEV), t.from_numpy(pos).to(DEV), y, T, H, D, 64, layout)
    t.cuda.synchronize()
    close(f64(y)[:, ok], ref, size, "far values")
    assert np.isnan(f64(y)[:, [3, 4]]).all()


@pytest.mark.gpu
def test_rope_strides_in_place_and_stream():
    t = torch()
    T, H, D = 21, 6, 128
    x, g, rng = heads(T, H, D, 3)
    pos, freq = rng.integers(0, 5000, T), FREQ(D)
    wide = t.full((T, H * D + 40), 3.0, dtype=t.bfloat16, device=DEV)
    wide[:, 16 : 16 + H * D] = x.view(T, -1).to(DEV)
    at = wide[:, 16 : 16 + H * D]
    s = t.cuda.Stream()
    args = t.from_numpy(freq).to(DEV), t.from_numpy(pos).to(DEV)
    gd = g.to(DEV)
    s.wait_stream(t.cuda.current_stream())
    sk.skgemm_rope(at, gd, *args, at, T, H, D, D, "half", stream=s)
    t.cuda.synchronize()
    ref, size = O.rope_ref(f64(x), f64(g), freq, pos, D, "half")
    close(f64(at).reshape(T, H, D), ref, size, "in place")
    assert (wide[:, :16] == 3).all() and (wide[:, 16 + H * D :] == 3).all()
    heads3 = wide[:, 16 : 16 + H * D].unflatten(1, (H, D))  # a 3-D view that is not contiguous
    y = t.empty(T, H, D, dtype=t.bfloat16, device=DEV)
    sk.skgemm_rope(heads3, None, None, None, y, T, H, D, 0)
    t.cuda.synchronize()
    assert t.equal(y, heads3)


def run_append(T, Hq, Hkv, D, rot, layout, page, fmt, order, norm, seed, k_scale=1.0, v_scale=1.0, slots=None, stream=None):
    """Outputs, references and what was there before; values of a split projection's rows."""
    t = torch()
    x, gq, rng = heads(T, Hq + 2 * Hkv, D, seed, spread=False)
    gk = bf16(1 + 0.2 * rng.standard_normal(D))
    pos, freq = rng.integers(0, 100000, T), FREQ(rot)
    n_pages = 2 * (-(-T // page)) + 1
    if slots is None:
        slots = rng.permutation(n_pages * page)[:T]
        slots[rng.random(T) < 0.1] = -1
        if T > 3:
            slots[1], slots[2] = n_pages * page, -(1 << 40)  # past the cache, far below it
    shape = (n_pages, page, Hkv, D) if order == "token" else (n_pages, Hkv, page, D)
    kind = t.uint8 if fmt == "e4m3" else t.bfloat16
    kc, vc = (t.full(shape, 0x31, dtype=t.uint8, device=DEV) if fmt == "e4m3" else t.full(shape, 5.5, dtype=kind, device=DEV) for _ in "kv")
    if order == "head":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    q_out = t.full((T, Hq * D), 7e7, dtype=t.bfloat16, device=DEV)
    row = x.view(T, -1).to(DEV)
    q, k, v = row.split((Hq * D, Hkv * D, Hkv * D), 1)
    up = lambda a: t.from_numpy(a).to(DEV)  # noqa: E731
    g = (gq.to(DEV), gk.to(DEV)) if norm else (None, None)
    args = up(freq), up(pos), up(slots.astype(np.int64))
    if stream is not None:
        stream.wait_stream(t.cuda.current_stream())
    sk.skgemm_rope_append(q, k, v, *g, *args, q_out, kc, vc, T, Hq, Hkv, D, n_pages, page, rot, layout, 1e-6, k_scale=k_scale,
                          v_scale=v_scale, stream=stream)
    t.cuda.synchronize()
    xf = f64(x)
    ref_q = O.rope_ref(xf[:, :Hq], f64(gq) if norm else None, freq, pos, rot, layout)
    ref_k = O.rope_ref(xf[:, Hq : Hq + Hkv], f64(gk) if norm else None, freq, pos, rot, layout)
    return q_out, kc, vc, slots, ref_q, ref_k, xf[:, Hq + Hkv :], n_pages * page


def check_append(out, T, Hq, Hkv, D, page, fmt, k_scale, v_scale):
    q_out, kc, vc, slots, (rq, sq), (rk, sk_), rv, n = out
    if Hq:
        close(f64(q_out).reshape(T, Hq, D), rq, sq, "queries")
    live = np.nonzero((slots >= 0) & (slots < n))[0]
    at = slots[live]
    raw = [c.contiguous().cpu() for c in (kc, vc)]
    if fmt == "e4m3":
        k, v = (a.numpy().reshape(n, Hkv, D) for a in raw)
        close_codes(k[at], rk[live], sk_[live], k_scale, "keys")
        close_codes(v[at], rv[live], np.abs(rv[live]), v_scale, "values")
    else:
        k, v = (f64(a).reshape(n, Hkv, D) for a in raw)
        close(k[at], rk[live], sk_[live], "keys")
        assert np.array_equal(v[at], rv[live])
    rest = np.setdiff1d(np.arange(n), at)
    old = 0x31 if fmt == "e4m3" else 5.5
    assert (k[rest] == old).all() and (v[rest] == old).all()  # nothing else was touched


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,layout,page,order,norm", [
    (1, 16, 2, 128, 128, "half", 16, "token", True), (67, 16, 2, 128, 128, "half", 16, "head", True),
    (5, 3, 1, 64, 32, "interleaved", 1, "token", False), (300, 14, 2, 64, 64, "half", 64, "head", True),
    (41, 8, 8, 256, 64, "half", 8, "token", False), (1100, 4, 2, 80, 80, "half", 32, "head", True),
    (13, 0, 5, 128, 128, "interleaved", 16, "token", True), (1030, 64, 8, 128, 128, "half", 128, "head", True),
])
def test_append(T, Hq, Hkv, D, rot, layout, page, order, norm, fmt):
    log(f"append T={T} Hq={Hq} Hkv={Hkv} D={D} rot={rot} {layout} page={page} {order} norm={norm} {fmt}")
    ks, vs = (0.11, 0.02) if fmt == "e4m3" else (1.0, 1.0)
    out = run_append(T, Hq, Hkv, D, rot, layout, page, fmt, order, norm, T + D, ks, vs)
    check_append(out, T, Hq, Hkv, D, page, fmt, ks, vs)


@pytest.mark.gpu
def test_append_saturates_and_keeps_nan():
    t = torch()
    D = 64
    k = t.zeros(1, D, dtype=t.bfloat16, device=DEV)
    v = k.clone()
    v[0, :6] = t.tensor([1e30, -1e30, float("nan"), float("inf"), 448.0, -500.0], device=DEV)
    kc = t.zeros(2, 1, 1, D, dtype=t.float8_e4m3fn, device=DEV)
    vc = t.zeros_like(kc)
    sk.skgemm_rope_append(None, k, v, None, None, None, None, t.tensor([1], device=DEV), None, kc, vc, 1, 0, 1, D, 2, 1, 0)
    t.cuda.synchronize()
    got = vc.float().cpu()[1, 0, 0]
    assert got[[0, 3, 4]].tolist() == [448.0] * 3 and got[[1, 5]].tolist() == [-448.0] * 2 and got[2].isnan()
    assert not vc.float()[0].any()


@pytest.mark.gpu
def test_append_captured_and_on_a_stream():
    t = torch()
    s = t.cuda.Stream()
    out = run_append(40, 4, 2, 128, 128, "half", 16, "bf16", "head", True, 1, stream=s)
    check_append(out, 40, 4, 2, 128, 16, "bf16", 1.0, 1.0)
    T, Hq, Hkv, D, n_pages = 17, 4, 2, 128, 4
    q, k, v = (t.randn(T, h * D, device=DEV).to(t.bfloat16) for h in (Hq, Hkv, Hkv))
    freq, pos, slots = t.from_numpy(FREQ(D)).to(DEV), t.arange(T, device=DEV), t.arange(T, device=DEV) + 20
    qo = t.empty_like(q)
    kc, vc = (t.zeros(n_pages, 16, Hkv, D, dtype=t.bfloat16, device=DEV) for _ in "kv")
    call = lambda: sk.skgemm_rope_append(q, k, v, None, None, freq, pos, slots, qo, kc, vc, T, Hq, Hkv, D, n_pages, 16, D)  # noqa: E731
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        call()
    for rep in range(3):
        pos += 1000 * rep
        slots.copy_(t.randperm(n_pages * 16, device=DEV)[:T])
        got = []
        for f in (g.replay, call):
            for a in (qo, kc, vc):
                a.zero_()
            f()
            t.cuda.synchronize()
            got.append([a.clone() for a in (qo, kc, vc)])
        assert all(t.equal(a, b) for a, b in zip(*got))


@pytest.mark.gpu
def test_rope_empty_calls():
    t = torch()
    x = t.zeros(0, 128, dtype=t.bfloat16, device=DEV)
    sk.skgemm_rope(x, None, None, None, x, 0, 1, 128, 0)
    sk.skgemm_rope_append(x, x, x, None, None, None, None, None, x, None, None, 0, 1, 1, 128, 0, 1, 0)


A = 1 << 20  # an address; every call below is refused before any is used


def test_rope_refusals():
    f = sk.lib().skgemm_rope

    def call(X=A, G=A, freq=A, pos=A, Y=2 * A, T=3, H=4, D=128, rot=64, layout=0, eps=1e-6, amp=1.0, xs=1024, ys=1024):
        return f(X, G, freq, pos, Y, T, H, D, rot, layout, eps, amp, xs, ys, None)

    assert call(T=-1) == call(H=-1) == call(rot=-16) == call(layout=2) == call(layout=-1) == sk.SKGEMM_EINVAL
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        assert call(eps=bad) == sk.SKGEMM_EINVAL
    assert call(amp=float("nan")) == call(amp=float("inf")) == sk.SKGEMM_EINVAL
    for D, rot in ((120, 64), (0, 0), (272, 64), (128, 24), (128, 144)):
        assert call(D=D, rot=rot) == sk.SKGEMM_ESHAPE
    assert call(H=4097) == call(T=(1 << 21) + 1) == sk.SKGEMM_ESHAPE
    assert call(X=None) == call(Y=None) == call(freq=None) == call(pos=None) == sk.SKGEMM_EINVAL
    assert call(X=A + 8) == call(Y=A + 8) == call(G=A + 2) == call(freq=A + 2) == call(pos=A + 4) == sk.SKGEMM_EALIGN
    assert call(xs=1032) == call(ys=1032) == sk.SKGEMM_EALIGN
    assert call(ys=1008) == call(Y=A, ys=2048) == sk.SKGEMM_EINVAL
    assert call(X=None, T=0) == call(X=None, H=0) == sk.SKGEMM_OK


def test_append_refusals():
    f = sk.lib().skgemm_rope_append

    def call(Q=A, K=A, V=A, Gq=A, Gk=A, freq=A, pos=A, slots=A, Qo=2 * A, KC=3 * A, VC=4 * A, T=3, Hq=4, Hkv=2, D=128, n=4, page=16,
             rot=64, layout=0, eps=1e-6, amp=1.0, fmt=0, ks=1.0, vs=1.0, qs=1024, kst=512, vst=512, qos=1024, ps=8192, ss=512, hs=256):
        return f(Q, K, V, Gq, Gk, freq, pos, slots, Qo, KC, VC, T, Hq, Hkv, D, n, page, rot, layout, eps, amp, fmt, ks, vs, qs, kst, vst,
                 qos, ps, ss, hs, None)

    for name in ("Q", "K", "V", "slots", "Qo", "KC", "VC", "freq", "pos"):
        assert call(**{name: None}) == sk.SKGEMM_EINVAL, name
        assert call(**{name: A + 2}) == sk.SKGEMM_EALIGN, name
    assert call(T=-1) == call(Hq=-1) == call(Hkv=-1) == call(n=0) == call(page=0) == call(fmt=1) == call(fmt=3) == sk.SKGEMM_EINVAL
    assert call(page=24) == call(page=1 << 16) == call(D=100) == sk.SKGEMM_ESHAPE
    assert call(ks=2.0) == call(vs=0.5) == call(fmt=2, ks=0.0) == call(fmt=2, vs=float("nan")) == call(fmt=2, ks=1e31) == sk.SKGEMM_EINVAL
    assert call(ps=8200) == call(ss=520) == call(hs=264) == call(qs=1032) == call(kst=520) == call(vst=520) == sk.SKGEMM_EALIGN
    # outputs on top of each other
    assert call(ss=256) == call(hs=128) == call(ps=4096) == call(ps=0) == call(hs=0) == call(KC=3 * A, VC=3 * A) == sk.SKGEMM_EINVAL
    assert call(Qo=A, qos=2048) == call(qos=512) == sk.SKGEMM_EINVAL
    assert call(ss=1 << 29) == call(hs=1 << 32) == call(ps=1 << 45) == sk.SKGEMM_ESHAPE
    assert call(T=0, Q=None) == call(Hq=0, Hkv=0) == sk.SKGEMM_OK


def test_rope_binding_refusals():
    t = torch()
    x = t.zeros(4, 128, dtype=t.bfloat16)
    for bad in (lambda: sk.skgemm_rope(x, None, None, None, A, 4, 1, 128, 0, stream=0),
                lambda: sk.skgemm_rope(A, None, None, None, A, 4, 1, 128, 0, layout="pairs", stream=0),
                lambda: sk.skgemm_rope(A, None, None, None, A, 4, 1, 128, 0, x_stride=-256, stream=0),
                lambda: sk.skgemm_rope_append(A, A, A, None, None, None, None, A, A, x.view(4, 1, 1, 128), A, 4, 1, 1, 128, 4, 1, 0, stream=0),
                lambda: sk.skgemm_rope_append(A, A, A, None, None, None, None, A, A, A, A, 4, 1, 1, 128, 4, 1, 0, cache_strides=(-256, 256, 256), stream=0),
                lambda: sk.skgemm_rope_append(A, A, A, None, None, None, None, A, A, A, A, 4, 1, 1, 128, 4, 1, 0, cache_format="int4", stream=0)):
        with pytest.raises(sk.SkgemmError) as e:
            bad()
        assert e.value.code == sk.SKGEMM_EINVAL
