"""skgemm_logprobs and skgemm_logprobs_grad against the fp64 formulas.

Bounds in units of u = 2^-24, with d = (x - max) scale / log 2, M1 = sum p |d|
and M2 = sum p d^2 of the row, n = the terms a thread adds up (a row over 256
threads at least):
* a term 2^d: three roundings in d (4 u |d| absolute), and one unit in the last
  place of the exponential (2 u); the sums: n additions of one sign, and fewer
  than 64 roundings where the threads' parts join. So
  log s is off by (n + 64 + 4 M1) u;
* lse: that, the product scale * max and the last addition: 6 u (|lse| + |scale max|);
* entropy = log s - sum p d: that twice, weighted: (n + 64)(1 + 2 M1) + 4 (M1 + M2 + M1^2)
  + 8 (|H| + 1) u;
* a log probability: log s, 6 u |d| and 4 u of itself;
* a gradient: log p is off by 3 u |log p|, p by (3 |log p| + 4) u of itself, the
  factor by 6 u of its parts, and bf16 rounds once more. Exponentials below
  FP32's normal range may be 0.
"""

import numpy as np
import pytest

import split_reduction_amd as sk
from oracle import ops as O
from tests.gpu_util import DEV, log, torch

U = O.EPS_F32


def dev_logits(z, kind, pad=0):
    t = torch()
    dt = t.float32 if kind == "f32" else t.bfloat16
    out = t.full((z.shape[0], z.shape[1] + pad), float("nan"), dtype=dt, device=DEV)
    out[:, : z.shape[1]] = t.from_numpy(z).to(DEV).to(dt)
    return out[:, : z.shape[1]]


def make(T, V, seed, banned=0.0, spread=2.5):
    rng = np.random.default_rng(seed)
    z = (spread * rng.standard_normal((T, V))).astype(np.float32)
    z[rng.random((T, V)) < banned] = -np.inf
    tok = rng.integers(0, V, T)
    z[np.arange(T), tok] = spread * rng.standard_normal(T) + 3
    return z, tok


def forward(Z, tok, k, scale, stream=None, want=("logprob", "entropy", "lse")):
    t = torch()
    T, V = Z.shape
    out = {n: t.full((T,), 77.0, device=DEV) for n in want}
    top, ids = t.full((T, k), 77.0, device=DEV), t.full((T, k), -7, dtype=t.int64, device=DEV)
    tk = t.from_numpy(np.asarray(tok, np.int64)).to(DEV)
    t.cuda.synchronize()
    sk.skgemm_logprobs(Z, tk, out.get("logprob"), out.get("entropy"), out.get("lse"), top if k else None,
                       ids if k else None, T, V, k, scale, stream=stream)
    t.cuda.synchronize()
    return {**{n: a.cpu().double().numpy() for n, a in out.items()}, "top": top.cpu().double().numpy(),
            "ids": ids.cpu().numpy()}


def near(got, want, tol, what):
    ok = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    same = ~ok & ~np.isnan(want)
    assert np.array_equal(got[same], want[same]), what
    worst = np.max((np.abs(got - want) / tol)[ok], initial=0.0)
    log(f"  {what}: largest error / bound {worst:.3f}")
    assert worst <= 1, what


def check_forward(Z, tok, k, scale, got=None):
    scale = float(np.float32(scale))  # as the call takes it
    raw = Z.double().cpu().numpy()
    tok = np.asarray(tok)
    got = forward(Z, tok, k, scale) if got is None else got
    with np.errstate(invalid="ignore", over="ignore"):
        ref = O.logprobs_ref(raw, tok, k, scale)
        n = -(-Z.shape[1] // (256 * 4)) * 8
        d = np.where(ref["p"] > 0, np.abs(ref["d"]), 0) / np.log(2)
        m1, m2 = (ref["p"] * d).sum(1), (ref["p"] * d * d).sum(1)
        s = (n + 64 + 4 * m1) * U
        near(got["lse"], ref["lse"], s + 6 * U * (np.abs(ref["lse"]) + np.abs(ref["m"])), "lse")
        near(got["entropy"], ref["entropy"],
             U * ((n + 64) * (1 + 2 * m1) + 4 * (m1 + m2 + m1**2) + 8 * (np.abs(ref["entropy"]) + 1)), "entropy")
        one = lambda v: s + U * (6 * np.abs(v + s) + 4 * np.abs(v) + 6 * np.abs(ref["lse"] - ref["m"]))  # noqa: E731
        near(got["logprob"], ref["logprob"], one(ref["logprob"]), "logprob")
        for i in range(k):
            assert np.array_equal(got["ids"][:, i], ref["ids"][:, i]), f"id {i}"
            near(got["top"][:, i], ref["top"][:, i], one(ref["top"][:, i]), f"top {i}")
    return got


SIZES = [(1, 1, 1), (1, 7, 7), (3, 8, 2), (2, 9, 1), (5, 100, 64), (1, 64, 64), (17, 1000, 5), (4, 2047, 20), (2, 2049, 64),
         (1, 32000, 20), (1, 131072, 20), (3, 131072, 1), (2, 262144, 64), (33, 50001, 8), (300, 4099, 3), (1, 1 << 20, 10),
         (600, 2500, 0), (2100, 1003, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,k", SIZES)
def test_logprobs(T, V, k, kind):
    z, tok = make(T, V, seed=T + V)
    log(f"logprobs T={T} V={V} k={k} {kind}")
    check_forward(dev_logits(z, kind), tok, k, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("scale", [0.7, 1.6])
def test_logprobs_strides_and_scale(kind, pad, scale):
    z, tok = make(21, 3001, seed=4, banned=0.5)
    tok[3], tok[5] = -1, -100
    check_forward(dev_logits(z, kind, pad), tok, 9, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 3001, 40000])
def test_logprobs_masks(V, kind):
    """Banned tokens, rows with fewer allowed tokens than alternatives asked for,
    one, none; the type's lowest value as a mask; equal logits; NaN and +inf."""
    t = torch()
    z, tok = make(16, V, seed=V)
    k = min(V, 30)
    low = float(t.finfo(t.float32 if kind == "f32" else t.bfloat16).min)
    z[0, 10:] = -np.inf
    z[1] = -np.inf
    z[1, V - 1] = 2.0
    z[2] = -np.inf
    z[3, 5:] = low
    z[4] = low
    z[5] = 0.25
    z[6] = -0.0
    z[6, V // 2:] = 0.0
    z[7, V // 3] = np.nan
    z[8, V // 2] = np.inf
    z[9] = -np.inf
    z[9, 3] = np.nan
    z[10, ::2] = z[10, 0]
    z[11] = np.linspace(30, -30, V)
    z[12] = np.linspace(-30, 30, V)
    z[13] = 1e4 + z[13]
    z[14] = -1e4 + z[14]
    tok[15] = V
    log(f"logprobs masks V={V} {kind}")
    check_forward(dev_logits(z, kind), tok, k, 1.0)


@pytest.mark.gpu
def test_logprobs_candidates_overflow():
    """The best tokens all with few owners: whole runs of vectors 256 apart hold
    them, so the candidates pass their buffer; and rows of one value."""
    V, k = 200000, 64
    for kind, per in (("bf16", 8), ("f32", 4)):
        z = np.full((3, V), -1.0, np.float32)
        j = np.arange(V) // per
        hot = (j % 256) < k
        rng = np.random.default_rng(1)
        z[0, hot] = 5 + rng.integers(0, 40, hot.sum())
        z[1, hot] = 5.0
        z[2] = 3.0
        log(f"logprobs overflow {kind}")
        check_forward(dev_logits(z, kind), [0, 1, 2], k, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 1200])
def test_logprobs_few_owners(T):
    """Fewer threads than alternatives hold all the large logits, thousands of
    them, distinct or equal: the candidates pass their buffer."""
    V, k = 200001, 64
    for kind, per in (("bf16", 8), ("f32", 4)):
        rng = np.random.default_rng(2)
        z = np.full((T, V), -1.0, np.float32)
        hot = (np.arange(V) // per) % 256 < 3
        z[0, hot] = 5 + rng.integers(0, 200, hot.sum()) / 8
        z[1, hot] = 5.0
        z[2:] = 3.0
        log(f"logprobs few owners {kind} T={T}")
        Z = dev_logits(z[:6], kind)
        if T > 6:  # the rows past the sixth equal it
            Z = torch().cat([Z, Z[5:].expand(T - 6, V)]).contiguous()
        tok = np.zeros(T, np.int64)
        got = forward(Z, tok, k, 1.0)
        for name, a in got.items():
            assert np.array_equal(a[6:], np.broadcast_to(a[5:6], a[6:].shape)) if T > 6 else True, name
        check_forward(Z[:6], tok[:6], k, 1.0, got={n: a[:6] for n, a in got.items()})


@pytest.mark.gpu
def test_logprobs_optional_outputs():
    z, tok = make(4, 500, seed=1)
    Z = dev_logits(z, "f32")
    full = check_forward(Z, tok, 4, 1.0)
    for want in (("lse",), ("entropy",), ("logprob",), ()):
        got = forward(Z, tok, 4, 1.0, want=want)
        for n in want + ("top", "ids"):
            assert np.array_equal(got[n], full[n]), n
    sk.skgemm_logprobs(Z, None, None, None, None, None, None, 4, 500)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(1, 131072), (3, 50001), (700, 3001)])
def test_logprobs_captured_and_streams(T, V):
    t = torch()
    k = 12
    z, tok = make(T, V, seed=2)
    Z, tk = dev_logits(z, "bf16"), t.from_numpy(tok).to(DEV)
    s, s2 = t.cuda.Stream(), t.cuda.Stream()

    def outs():
        return [t.zeros(T, device=DEV) for _ in range(3)] + [t.zeros(T, k, device=DEV), t.zeros(T, k, dtype=t.int64, device=DEV)]

    a, b, c = outs(), outs(), outs()
    t.cuda.synchronize()
    for _ in range(3):
        sk.skgemm_logprobs(Z, tk, *a, T, V, k, stream=s)
        sk.skgemm_logprobs(Z, tk, *b, T, V, k, stream=s2)
    t.cuda.synchronize()
    assert all(t.equal(x, y) for x, y in zip(a, b))
    check_forward(Z, tok, k, 1.0, got=dict(zip(("logprob", "entropy", "lse", "top", "ids"), (
        x.cpu().double().numpy() if x.is_floating_point() else x.cpu().numpy() for x in a))))
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr, stream=s):
        sk.skgemm_logprobs(Z, tk, *c, T, V, k, stream=s)
    for _ in range(3):
        for x in c:
            x.zero_()
        t.cuda.synchronize()
        with t.cuda.stream(s):
            gr.replay()
        t.cuda.synchronize()
        assert all(t.equal(x, y) for x, y in zip(a, c))
        sk.skgemm_logprobs(Z, tk, *b, 1, 1000, k, stream=s)
        t.cuda.synchronize()


# ---- the gradient ----


def backward(Z, tok, lse, ent, g, gh, scale, D=None):
    t = torch()
    T, V = Z.shape
    up = lambda a: None if a is None else t.from_numpy(np.asarray(a, np.float32)).to(DEV)  # noqa: E731
    D = t.full_like(Z, 55.0) if D is None else D
    dev = [up(a) for a in (lse, ent, g, gh)]
    tk = None if tok is None else t.from_numpy(np.asarray(tok, np.int64)).to(DEV)
    t.cuda.synchronize()
    sk.skgemm_logprobs_grad(Z, tk, *dev, D, T, V, scale)
    t.cuda.synchronize()
    return D.double().cpu().numpy()


def check_backward(Z, tok, scale, seed=0, use=("g", "gh"), D=None, kind="f32"):
    scale = float(np.float32(scale))  # as the call takes it
    rng = np.random.default_rng(seed)
    T, V = Z.shape
    raw = Z.double().cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        f = O.logprobs_ref(raw, np.asarray(tok), 0, scale)
        lse, ent = f["lse"].astype(np.float32), f["entropy"].astype(np.float32)
        g = rng.standard_normal(T).astype(np.float32) if "g" in use else None
        gh = (0.3 * rng.standard_normal(T)).astype(np.float32) if "gh" in use else None
        got = backward(Z, tok if g is not None else None, lse, ent if gh is not None else None, g, gh, scale, D)
        z32 = np.zeros(T, np.float32)
        g, gh = (z32 if g is None else g).astype(np.float64), (z32 if gh is None else gh).astype(np.float64)
        h = ent.astype(np.float64)
        want, p, lp = O.logprobs_grad_ref(raw, np.asarray(tok), lse.astype(np.float64), h, g, gh, scale)
        past = (np.asarray(tok) >= V) & ("g" in use)
        want[past | np.isnan(lse)] = np.nan
        parts = np.abs(g)[:, None] + np.abs(gh)[:, None] * (np.abs(h)[:, None] + np.abs(lp))
        tol = U * scale * p * ((3 * np.abs(lp) + 4) * parts + 6 * parts) + 4 * U * scale * np.abs(g)[:, None] * (
            np.arange(V) == np.asarray(tok)[:, None]) + 1e-36 * scale * (1 + parts)
        if kind == "bf16":
            tol = tol * (1 + O.EPS_BF16) + O.EPS_BF16 * np.abs(want)
        near(got, want, tol, "gradient")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (1, 9), (3, 8), (5, 100), (17, 1000), (4, 2047), (1, 131072), (33, 50001), (300, 4099),
                                 (2100, 1003), (1, 1 << 20)])
def test_logprobs_grad(T, V, kind):
    z, tok = make(T, V, seed=T + V)
    log(f"logprobs grad T={T} V={V} {kind}")
    check_backward(dev_logits(z, kind), tok, 1.0, kind=kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("use", [("g", "gh"), ("g",), ("gh",)])
def test_logprobs_grad_masks_strides_in_place(kind, use):
    """Banned tokens, empty rows, padding, rows of another alignment than the
    gradient's, and the gradient on top of the logits."""
    t = torch()
    z, tok = make(12, 3001, seed=9, banned=0.5)
    z[1] = -np.inf
    z[2, 7:] = float(t.finfo(t.float32 if kind == "f32" else t.bfloat16).min)
    tok[2] = 3
    z[3, 5] = np.nan
    tok[4], tok[5] = -1, 3001
    for pad, dpad in ((0, 0), (1, 1), (3, 0), (2, 5)):
        Z = dev_logits(z, kind, pad)
        D = t.full((12, 3001 + dpad), 55.0, dtype=Z.dtype, device=DEV)
        check_backward(Z, tok, 1.3, use=use, D=D[:, :3001], kind=kind)
        assert (D[:, 3001:] == 55).all()
    Z = dev_logits(z, kind, 0)
    up = lambda a: t.from_numpy(np.asarray(a, np.float32)).to(DEV)  # noqa: E731
    f = forward(Z, tok, 0, 1.3)
    args = (t.from_numpy(tok).to(DEV), up(f["lse"]), up(f["entropy"]), up(np.ones(12)), up(np.ones(12)))
    D = t.empty_like(Z)
    sk.skgemm_logprobs_grad(Z, *args, D, 12, 3001, 1.3)
    sk.skgemm_logprobs_grad(Z, *args, Z, 12, 3001, 1.3)
    t.cuda.synchronize()
    assert t.equal(Z.nan_to_num(9.0), D.nan_to_num(9.0))


def test_gradient_formula_against_differences():
    """The fp64 formula that the kernel is held to, against central differences
    of the fp64 forward."""
    rng = np.random.default_rng(3)
    z, tok = make(3, 11, seed=3)
    z[1, 4] = -np.inf
    tok[1] = 2
    tok[2] = -1
    z = z.astype(np.float64)
    scale, g, gh = 1.4, rng.standard_normal(3), rng.standard_normal(3)

    def loss(a):
        f = O.logprobs_ref(a, tok, 0, scale)
        return g * f["logprob"] + gh * f["entropy"]

    f = O.logprobs_ref(z, tok, 0, scale)
    d, _, _ = O.logprobs_grad_ref(z, tok, f["lse"], f["entropy"], g, gh, scale)
    h = 1e-6
    for j in range(11):
        e = np.zeros_like(z)
        e[:, j] = h
        num = (loss(z + e) - loss(z - e)) / (2 * h)
        live = np.isfinite(z[:, j])
        assert np.allclose(d[live, j], num[live], atol=2e-8), j
        assert np.all(d[~live, j] == 0)


def test_reference_against_library_routines():
    t = torch()
    z, tok = make(7, 300, seed=1, banned=0.3)
    f = O.logprobs_ref(z, tok, 5, 0.8)
    a = t.from_numpy(z).double() * 0.8
    lp = t.log_softmax(a, 1)
    assert np.allclose(f["lse"], t.logsumexp(a, 1).numpy(), atol=1e-12)
    assert np.allclose(f["entropy"], t.special.entr(lp.exp()).sum(1).numpy(), atol=1e-12)
    assert np.allclose(f["logprob"], lp[t.arange(7), t.from_numpy(tok)].numpy(), atol=1e-12)
    assert np.allclose(f["top"], t.topk(lp, 5).values.numpy(), atol=1e-12)


def test_logprobs_refusals():
    f, b = sk.lib().skgemm_logprobs, sk.lib().skgemm_logprobs_grad
    a = 1 << 20

    def call(z=a, tok=a, lp=a, ent=a, lse=a, tv=a, ti=a, T=2, V=32, k=4, scale=1.0, fmt=0, st=64):
        return f(z, tok, lp, ent, lse, tv, ti, T, V, k, scale, fmt, st, None)

    def grad(z=a, tok=a, lse=a, ent=a, g=a, gh=a, d=a << 1, T=2, V=32, scale=1.0, fmt=0, st=64, ds=64):
        return b(z, tok, lse, ent, g, gh, d, T, V, scale, fmt, st, ds, None)

    for c in (call, grad):
        assert c(T=-1) == c(V=-1) == c(fmt=1) == c(fmt=2) == c(z=None) == sk.SKGEMM_EINVAL
        for bad in (0.0, -1.0, float("nan"), float("inf")):
            assert c(scale=bad) == sk.SKGEMM_EINVAL
        assert c(V=(1 << 20) + 1, st=1 << 22) == c(T=(1 << 21) + 1) == sk.SKGEMM_ESHAPE
        assert c(z=a + 8) == c(st=65) == c(tok=a + 4) == c(lse=a + 2) == sk.SKGEMM_EALIGN
        assert c(st=62) == sk.SKGEMM_EINVAL
        assert c(z=None, T=0) == c(z=None, V=0) == sk.SKGEMM_OK
    assert call(k=-1) == call(k=33) == call(tok=None) == call(tv=None) == call(ti=None) == sk.SKGEMM_EINVAL
    assert call(k=65, V=100, st=200) == sk.SKGEMM_ESHAPE
    assert call(ti=a + 4) == call(tv=a + 2) == call(lp=a + 2) == call(ent=a + 2) == sk.SKGEMM_EALIGN
    assert grad(tok=None) == grad(ent=None) == grad(lse=None) == grad(d=None) == sk.SKGEMM_EINVAL
    assert grad(ds=62) == grad(d=a, ds=128) == sk.SKGEMM_EINVAL
    assert grad(d=(a << 1) + 8) == grad(ds=65) == grad(g=a + 2) == grad(gh=a + 2) == sk.SKGEMM_EALIGN


def test_logprobs_binding_refusals():
    t = torch()
    for call in (lambda z: sk.skgemm_logprobs(z, 1 << 20, 1 << 20, None, None, None, None, 2, 32),
                 lambda z: sk.skgemm_logprobs_grad(z, 1 << 20, 1 << 20, 1 << 20, 1 << 20, None, 1 << 20, 2, 32)):
        with pytest.raises(sk.SkgemmError) as e:
            call(t.zeros(2, 32))
        assert e.value.code == sk.SKGEMM_EINVAL and "not on the GPU" in str(e.value)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(3, 131072), (64, 131072), (300, 50001), (700, 40000)])
@pytest.mark.parametrize("k", [20, 64])
def test_logprobs_rows_of_many_nan(T, V, k, kind):
    """NaN among banned logits, among ordinary ones, and alone, in rows that are
    split and rows that are not; the other rows keep their results."""
    t = torch()
    z, tok = make(6, V, seed=V + k)
    rng = np.random.default_rng(k)
    z[0, rng.random(V) < 0.5] = -np.inf
    z[0, np.isfinite(z[0])] = np.nan
    z[1, ::2] = np.nan
    z[2] = np.nan
    z[3] = -np.inf
    z[3, V - V // 40 :: 3] = np.nan  # in a split row's last runs
    z[4, ::2] = -np.inf
    rows = np.resize(np.arange(6), T)
    log(f"logprobs many NaN T={T} V={V} k={k} {kind}")
    Z = dev_logits(z, kind)[t.from_numpy(rows).to(DEV)].contiguous()
    got = forward(Z, tok[rows], k, 1.0)
    n = min(T, 24)  # past these, rows and their alignments repeat
    for name, a in got.items():
        assert np.array_equal(a, a[np.arange(T) % 24], equal_nan=True), name
    check_forward(Z[:n], tok[rows][:n], k, 1.0, got={name: a[:n] for name, a in got.items()})


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale,weight", [(1.0, 3e9), (256.0, 1e7), (0.5, 1e30)])
def test_logprobs_grad_large_weights(kind, scale, weight):
    """Banned tokens, and tokens far below the best, under large weights of the
    entropy: zeros, not 0 * inf. The bound is check_backward's."""
    t = torch()
    T, V = 5, 3001
    z, tok = make(T, V, seed=3, banned=0.5)
    z[1, 7:] = float(t.finfo(t.float32 if kind == "f32" else t.bfloat16).min)
    z[2] = -np.inf
    z[2, [4, 9]] = 1.0, 1.5
    tok[1], tok[2] = 3, 4
    Z = dev_logits(z, kind)
    raw = Z.double().cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        f = O.logprobs_ref(raw, tok, 0, scale)
        lse, ent = f["lse"].astype(np.float32), f["entropy"].astype(np.float32)
        g, gh = np.full(T, weight, np.float32), np.linspace(-weight, weight, T).astype(np.float32)
        got = backward(Z, tok, lse, ent, g, gh, scale)
        h, g, gh = (a.astype(np.float64) for a in (ent, g, gh))
        want, p, lp = O.logprobs_grad_ref(raw, tok, lse.astype(np.float64), h, g, gh, scale)
    parts = np.abs(g)[:, None] + np.abs(gh)[:, None] * (np.abs(h)[:, None] + np.abs(lp))
    tol = U * scale * p * ((3 * np.abs(lp) + 4) * parts + 6 * parts) + 4 * U * scale * np.abs(g)[:, None] * (
        np.arange(V) == tok[:, None]) + 1e-36 * scale * (1 + parts)
    if kind == "bf16":
        tol = tol * (1 + O.EPS_BF16) + O.EPS_BF16 * np.abs(want)
    assert np.all(got[~np.isfinite(z)] == 0)
    near(got, want, tol, "gradient")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e10, 2e38])
def test_logprobs_near_zero_temperature(kind, scale):
    """All probability with the best token, shared where it is not alone."""
    V = 3001
    z, tok = make(4, V, seed=6)
    z = np.round(z * 4) / 4  # apart by 1/4 or equal
    z[1, [5, 900]] = z[1].max() + 1
    tok[1] = 900
    z[2] = 0.0
    z[3, 1:] = -np.inf
    tok[3] = 0
    Z = dev_logits(z, kind)
    got = forward(Z, tok, 3, scale)
    n = (z == z.max(1, keepdims=True)).sum(1)
    assert np.allclose(got["entropy"], np.log(n), rtol=1e-6, atol=0)
    assert np.allclose(got["logprob"][1:], -np.log(n[1:]), rtol=1e-6, atol=0)
    best = np.argsort(-z, axis=1, kind="stable")[:, :3]
    assert np.array_equal(got["ids"], best)
    assert np.allclose(got["top"][:, 0], -np.log(n), rtol=1e-6, atol=0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_logprobs_scaled_past_the_range(kind):
    """scale * max past FP32's range: an infinite lse, the other outputs right. The
    gradient has no probabilities to work with: NaN, or zeros where lse is -inf."""
    t = torch()
    V = 1000
    z = np.zeros((2, V), np.float32)
    z[0, :7], z[0, 7:] = 3e38, 1e38
    z[1] = -3e38
    tok = np.array([3, 8])
    Z = dev_logits(z, kind)
    got = forward(Z, tok, 2, 2.0)
    n = np.array([7, V])
    assert np.array_equal(got["lse"], [np.inf, -np.inf])
    for a in (got["entropy"], -got["logprob"], -got["top"][:, 0], -got["top"][:, 1]):
        assert np.allclose(a, np.log(n), rtol=1e-6, atol=0)
    assert np.array_equal(got["ids"], [[0, 1], [0, 1]])
    d = backward(Z, tok, got["lse"], got["entropy"], np.ones(2), np.ones(2), 2.0)
    assert np.isnan(d[0]).all() and not d[1].any()
