"""skgemm_paged_attention against the fp64 formula, and its refusals.

Bounds, with e = 2^-24 and what a row sees: S = the largest scale * sum |q_i k_i|,
A = sum p |v|, N tokens:
* a score's products are exact in FP32 and summed in D additions; scale, its product
  with k_scale and the step to powers of two 4 more: off by d = S (D + 4) e;
* a probability: exp of two scores off by d each, the subtraction's rounding 2 S e and
  2 of the exponential, N + 64 for the sum and the joins' rescalings, the rounding to
  bf16 2^-8: together 2 d + 2 S e + (N + 66) e + 2^-8;
* O: A times that and N + 64 + 3 (FP32 sums, joins, division, v_scale) e, and one bf16
  rounding of the result, and 2^-133 where that is below the smallest normal;
* lse: d + 2 S e, (N + 66) e of the sum, and 4 roundings of its own size.
Every slot of the cache that no token owns holds NaN.
"""

import numpy as np
import pytest

import split_reduction_amd as sk
from oracle import ops as O
from tests.gpu_util import DEV, log, torch

E = O.EPS_F32


def f64(a):
    return a.float().double().cpu().numpy()


class Case:
    """Sequences of (new, all) tokens, their cache and its table."""

    def __init__(self, seqs, Hkv=2, G=4, D=128, page=16, fmt="bf16", order="head", pad=0, before=0, seed=0, q_size=2.0, extra_pages=3):
        t = torch()
        rng = np.random.default_rng(seed)
        self.seqs, self.Hkv, self.Hq, self.D, self.page, self.fmt = seqs, Hkv, G * Hkv, D, page, fmt
        self.B, self.before = len(seqs), before
        self.ks, self.vs = (0.07, 0.03) if fmt == "e4m3" else (1.0, 1.0)
        starts = before + np.concatenate([[0], np.cumsum([n for n, _ in seqs])])
        self.T = int(starts[-1]) + pad
        need = [-(-L // page) for _, L in seqs]
        self.max_pages = max(need + [1]) + 1
        self.n_pages = sum(need) + extra_pages
        ids = rng.permutation(self.n_pages)
        self.table = np.full((self.B, self.max_pages), -7, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = ids[at : at + k]
            at += k
        shape = (self.n_pages, page, Hkv, D)
        nan = t.tensor(float("nan"))
        mem = shape if order == "token" else (shape[0], Hkv, page, D)
        kind = t.float8_e4m3fn if fmt == "e4m3" else t.bfloat16
        cache = []
        self.values = []  # [L, Hkv, D] of each sequence, as stored
        for size, scale in ((1.0, self.ks), (1.0, self.vs)):
            c = nan.expand(mem).to(kind).clone()
            view = c if order == "token" else c.transpose(1, 2)
            stored = []
            for b, (n, L) in enumerate(seqs):
                x = t.from_numpy((size * rng.standard_normal((L, Hkv, D)) / scale).astype(np.float32)).to(kind)
                for p in range(need[b]):
                    m = min(page, L - p * page)
                    view[self.table[b, p], :m].view(t.uint8 if fmt == "e4m3" else t.bfloat16).copy_(
                        x[p * page : p * page + m].view(t.uint8 if fmt == "e4m3" else t.bfloat16))
                stored.append(x)
            cache.append(c)
            self.values.append(stored)
        self.mem = [c.to(DEV) for c in cache]
        self.kc, self.vc = (c if order == "token" else c.transpose(1, 2) for c in self.mem)
        self.q = t.from_numpy((q_size * rng.standard_normal((self.T, self.Hq, D))).astype(np.float32)).to(t.bfloat16)
        i32 = lambda a: t.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
        self.table_d, self.start_d, self.len_d = i32(self.table), i32(starts), i32([L for _, L in seqs])
        self.starts = starts
        self.qd = self.q.to(DEV)
        self.max_q = max([n for n, _ in seqs])

    def call(self, o, lse, window=0, max_q=None, q=None, **kw):
        sk.skgemm_paged_attention(self.qd if q is None else q, self.kc, self.vc, self.table_d, self.len_d, self.start_d, o, lse, self.T,
                                  self.B, self.max_q if max_q is None else max_q, self.Hq, self.Hkv, self.D, self.n_pages, self.page,
                                  self.max_pages, self.D**-0.5, window, self.ks, self.vs, **kw)

    def run(self, window=0, **kw):
        t = torch()
        o = t.full((self.T, self.Hq, self.D), 7.75, dtype=t.bfloat16, device=DEV)
        lse = t.full((self.T, self.Hq), -55.0, device=DEV)
        self.call(o, lse, window, **kw)
        t.cuda.synchronize()
        return o, lse

    def check(self, o, lse, window=0, rows=None):
        """Of each sequence all rows, or those that rows(n) gives."""
        got, glse = f64(o), lse.double().cpu().numpy()
        worst = 0.0
        for b, (n, L) in enumerate(self.seqs):
            if n == 0:
                continue
            a = int(self.starts[b])
            pick = list(range(n)) if rows is None else rows(n)
            k = f64(self.values[0][b]) * self.ks
            v = f64(self.values[1][b]) * self.vs
            for i in pick:
                p = L - n + i
                q = f64(self.q[a + i : a + i + 1])
                ref, rl, A, S = O.attention_ref(q, k[: max(p + 1, 0)], v[: max(p + 1, 0)], self.D**-0.5, window) if p >= 0 else (
                    np.zeros((1, self.Hq, self.D)), np.full((1, self.Hq), -np.inf), 0.0, np.zeros((1, self.Hq)))
                g, gl = got[a + i], glse[a + i]
                if p < 0:
                    assert (g == 0).all() and np.isneginf(gl).all(), (b, i)
                    continue
                N = min(p + 1, window) if window else p + 1
                d = S[0] * (self.D + 4) * E
                soft = 2 * d + 2 * S[0] * E + (N + 66) * E
                tol = A[0] * (soft + O.EPS_BF16 + (N + 67) * E)[:, None] * (1 + O.EPS_BF16) + O.EPS_BF16 * np.abs(ref[0]) + 2.0**-133
                ratio = np.abs(g - ref[0]) / tol
                tl = d + 2 * S[0] * E + (N + 66) * E + 4 * E * np.abs(rl[0])
                worst = max(worst, float(ratio.max()), float((np.abs(gl - rl[0]) / tl).max()))
                assert np.isfinite(g).all() and ratio.max() <= 1, (b, i, n, L, float(ratio.max()))
                assert np.all(np.abs(gl - rl[0]) <= tl), (b, i, n, L)
        used = np.zeros(self.T, bool)
        used[self.before : int(self.starts[-1])] = True
        assert (got[~used] == 7.75).all() and (glse[~used] == -55).all()  # padding is left alone
        log(f"  largest error / bound {worst:.3f}")


SINGLE = [(1, 1), (1, 2), (1, 31), (1, 32), (1, 33), (1, 127), (1, 128), (1, 129), (1, 257), (1, 1000), (1, 5)]
MIXED = [(5, 5), (1, 40), (33, 33), (64, 200), (0, 0), (100, 357), (1, 1), (0, 50), (2, 700), (17, 64), (3, 129)]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,order,G,Hkv", [(16, "head", 8, 1), (1, "token", 1, 3), (64, "token", 7, 2), (256, "head", 32, 1)])
def test_single_tokens(D, fmt, page, order, G, Hkv):
    c = Case(SINGLE, Hkv, G, D, page, fmt, order, pad=2, before=1, seed=D + page)
    log(f"attention single tokens D={D} {fmt} page={page} {order} G={G} Hkv={Hkv}")
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,order,G,Hkv", [(16, "token", 4, 2), (8, "head", 7, 1), (128, "head", 1, 2), (2, "token", 40, 1)])
def test_chunks_and_single_tokens(D, fmt, page, order, G, Hkv):
    c = Case(MIXED, Hkv, G, D, page, fmt, order, pad=3, seed=D + G)
    log(f"attention mixed D={D} {fmt} page={page} {order} G={G} Hkv={Hkv}")
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("D,fmt", [(64, "bf16"), (128, "bf16"), (128, "e4m3"), (256, "bf16"), (256, "e4m3"), (64, "e4m3")])
@pytest.mark.parametrize("seqs", [[(n, n)] for n in (1, 2, 63, 64, 65, 300)] + [[(8, 5)], [(70, 40)], [(2, 0)], [(90, 0)]])
def test_one_sequence(seqs, D, fmt):
    """Prompts of all lengths; more new tokens than tokens: rows that see nothing."""
    c = Case(seqs, 2, 4, D, 16, fmt, "head", pad=1, seed=seqs[0][0])
    log(f"attention {seqs} D={D} {fmt}")
    c.check(*c.run(), rows=lambda n: sorted({0, 1, n // 2, n - 1} & set(range(n))) if n > 70 else range(n))


@pytest.mark.gpu
@pytest.mark.parametrize("D,fmt", [(128, "bf16"), (64, "e4m3"), (256, "bf16")])
@pytest.mark.parametrize("seqs,G", [([(1, 20000)], 8), ([(1, 9000), (1, 3), (1, 700)], 3), ([(300, 6000)], 4), ([(40, 5000), (1, 3000)], 2),
                                    ([(4, 12345)], 8), ([(1, 100)] * 70 + [(1, 5000)], 1)])
def test_long(seqs, G, D, fmt):
    """Keys split over workgroups and joined."""
    c = Case(seqs, 1, G, D, 32, fmt, "head", seed=G)
    log(f"attention long {seqs[-1]} D={D} {fmt}")
    c.check(*c.run(), rows=lambda n: sorted({0, n // 3, n - 1}))


@pytest.mark.gpu
@pytest.mark.parametrize("D,fmt", [(64, "bf16"), (64, "e4m3"), (128, "bf16"), (128, "e4m3"), (256, "bf16")])
@pytest.mark.parametrize("G,Hkv,window", [(4, 2, 0), (1, 3, 0), (16, 1, 0), (7, 1, 3000)])
def test_chunks_over_long_caches(D, fmt, G, Hkv, window):
    """Batches whose keys are split, beside sequences of few rows that are split as well."""
    c = Case([(70, 5000), (1, 6100), (0, 40), (300, 301), (33, 4097), (1, 1), (5, 2049), (129, 100)], Hkv, G, D, 16, fmt, "head", pad=1, seed=D + G)
    log(f"attention chunks over long caches D={D} {fmt} G={G} Hkv={Hkv} window={window}")
    c.check(*c.run(window), window, rows=lambda n: sorted({0, n // 3, n - 1}))


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 16, 100, 2000, 2**31 - 1])
@pytest.mark.parametrize("D,fmt", [(128, "bf16"), (64, "e4m3"), (256, "e4m3")])
def test_window(window, D, fmt):
    c = Case([(1, 1500), (60, 300), (1, 17), (130, 130), (2, 64), (9, 4), (1, 0)], 2, 3, D, 16, fmt, "token", pad=1, seed=window % 97)
    log(f"attention window={window} D={D} {fmt}")
    c.check(*c.run(window), window, rows=lambda n: range(0, n, 1 if n < 20 else 7))


@pytest.mark.gpu
def test_batches_past_a_wave():
    """More sequences than lanes, some without rows."""
    rng = np.random.default_rng(5)
    seqs = [(int(n), int(n + L)) for n, L in zip(rng.choice([0, 1, 1, 1, 3, 40], 200), rng.integers(0, 150, 200))]
    c = Case(seqs, 1, 2, 64, 16, "bf16", "head", seed=6)
    c.check(*c.run(), rows=lambda n: sorted({0, n - 1}))


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D,fmt", [(128, "bf16"), (64, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_not_finite_where_a_row_does_not_look(D, fmt, bad):
    """Keys and values that are no numbers leave the rows alone that do not see them;
    of those that do, a value's output is lost, a key's whole row."""
    t = torch()
    if fmt == "e4m3":
        bad = float("nan")
    for seqs, where, window in (([(40, 100)], 80, 0), ([(3, 70)], 68, 0), ([(40, 100)], 50, 20), ([(300, 300)], 130, 0), ([(1, 90)], 30, 40)):
        n, L = seqs[0]
        for which in (0, 1):
            c = Case(seqs, 1, 4, D, 16, fmt, "token", seed=where)
            clean = c.run(window)
            c.check(*clean, window, rows=lambda n: sorted({0, n - 1}))
            page, slot = int(c.table[0, where // 16]), where % 16
            (c.kc, c.vc)[which][page, slot, 0, 5] = t.tensor(bad).to(c.kc.dtype)
            o, lse = c.run(window)
            place = L - n + np.arange(n)
            sees = (place >= where) & ((place - where < window) if window else True)
            a, b = f64(o), f64(clean[0])
            assert np.array_equal(a[~sees], b[~sees]) and t.equal(lse.cpu()[~sees], clean[1].cpu()[~sees]), (seqs, which)
            if which == 1:
                keep = np.arange(D) != 5
                assert not np.isfinite(a[sees][:, :, 5]).any()
                assert np.array_equal(a[sees][:, :, keep], b[sees][:, :, keep]) and t.equal(lse, clean[1])
            elif np.isnan(bad) and sees.any():
                assert np.isnan(a[sees]).all()


@pytest.mark.gpu
def test_bad_pages_are_not_read():
    """Ids past the cache or below 0: the rows that see them are NaN, other sequences are right."""
    t = torch()
    for seqs in ([(1, 100), (1, 100)], [(80, 100), (80, 100)], [(1, 6000), (1, 100)]):
        for bad in (-1, 1 << 30, None):
            c = Case(seqs, 2, 4, 128, 16, "bf16", "head", seed=1)
            c.table_d[0, 2] = c.n_pages if bad is None else bad
            o, lse = c.run()
            n = seqs[0][0]
            sees = seqs[0][1] - n + np.arange(n) >= 32
            assert np.isnan(f64(o[:n])[sees]).all() and np.isnan(lse[:n].cpu().numpy()[sees]).all()
            c.seqs = [(0, 0), c.seqs[1]]
            c.before = n
            got = o.clone()
            got[:n] = 7.75
            lse[:n] = -55
            c.check(got, lse, rows=lambda n: sorted({0, n - 1}))
    c = Case([(4, 30)], 1, 2, 64, 16, "bf16", "head", seed=2)  # lengths and starts outside their arrays
    c.len_d[0] = 1 << 30
    c.run()
    c.len_d[0] = -5
    o, lse = c.run()
    assert (f64(o) == 0).all() and np.isneginf(lse.cpu().numpy()).all()
    c.start_d.copy_(t.tensor([2, 1 << 30], dtype=t.int32))
    c.len_d[0] = 30
    o, _ = c.run()
    assert (f64(o[:2]) == 7.75).all() and np.isfinite(f64(o)).all()
    c.start_d.copy_(t.tensor([3, -9], dtype=t.int32))
    o, _ = c.run()
    assert (f64(o) == 7.75).all()


@pytest.mark.gpu
def test_large_scores():
    """Maxima that grow from tile to tile, equal scores, and scores far apart."""
    t = torch()
    c = Case([(1, 700), (40, 700)], 1, 4, 128, 16, "bf16", "token", seed=3)
    for b in range(2):
        k = f64(c.values[0][b])
        k *= np.linspace(0, 40, 700)[:, None, None]
        k = t.from_numpy(k.astype(np.float32)).to(t.bfloat16)
        c.values[0][b] = k
        for p in range(-(-700 // 16)):
            m = min(16, 700 - 16 * p)
            c.kc[c.table[b, p], :m] = k[16 * p : 16 * p + m].to(DEV)
    c.check(*c.run(), rows=lambda n: sorted({0, 7, n - 1} & set(range(n))))
    c.qd.zero_()
    c.q.zero_()
    c.check(*c.run(), rows=lambda n: sorted({0, n - 1}))


@pytest.mark.gpu
@pytest.mark.parametrize("seqs", [[(1, 300), (1, 2000)], [(70, 90), (1, 33)]])
def test_strides_in_place_and_stream(seqs):
    """Q inside a wider product's rows, O on top of Q, a sliced table, another stream."""
    t = torch()
    c = Case(seqs, 2, 4, 64, 16, "bf16", "token", seed=8)
    want, wl = c.run()
    HD = c.Hq * c.D
    row = t.full((c.T, HD + 256), 3.0, dtype=t.bfloat16, device=DEV)
    row[:, 128 : 128 + HD] = c.qd.view(c.T, -1)
    table = t.full((c.B, c.max_pages + 5), -1, dtype=t.int32, device=DEV)
    table[:, 2 : 2 + c.max_pages] = c.table_d
    c.table_d = table[:, 2 : 2 + c.max_pages]
    at = row[:, 128 : 128 + HD]
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    lse = t.empty(c.T, c.Hq, device=DEV)
    c.call(at, lse, q=at, stream=s)
    t.cuda.synchronize()
    assert t.equal(at, want.view(c.T, -1)) and t.equal(lse, wl)
    assert (row[:, :128] == 3).all() and (row[:, 128 + HD :] == 3).all()
    o = t.empty(c.T, c.Hq, c.D, dtype=t.bfloat16, device=DEV)
    c.call(o, None)  # without lse
    t.cuda.synchronize()
    assert t.equal(o, want)


@pytest.mark.gpu
def test_same_bits_every_time():
    c = Case([(1, 5000), (1, 4000), (100, 3000)], 2, 4, 128, 16, "bf16", "head", seed=4)
    first = c.run()
    for _ in range(4):
        again = c.run()
        assert all(torch().equal(a, b) for a, b in zip(first, again))


@pytest.mark.gpu
def test_captured_with_other_lengths():
    """A graph captured once serves other lengths and tables; eager calls between."""
    t = torch()
    c = Case([(1, 900), (1, 1500), (40, 700)], 2, 4, 128, 16, "bf16", "head", seed=12)
    o = t.empty(c.T, c.Hq, c.D, dtype=t.bfloat16, device=DEV)
    lse = t.empty(c.T, c.Hq, device=DEV)
    s = t.cuda.Stream()
    sk.skgemm_reserve_ops(s)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        c.call(o, lse, stream=s)
    for lens in ([900, 1500, 700], [1, 1400, 40], [16, 17, 650]):
        c.len_d.copy_(t.tensor(lens, dtype=t.int32))
        t.cuda.synchronize()
        with t.cuda.stream(s):
            o.zero_()
            g.replay()
        t.cuda.synchronize()
        want, wl = c.run()
        assert t.equal(o, want) and t.equal(lse, wl)
    del g


@pytest.mark.gpu
def test_two_streams_at_once():
    t = torch()
    cases = [Case([(1, 3000), (1, 2500)], 2, 4, 128, 16, "bf16", "head", seed=s) for s in (1, 2)]
    want = [c.run() for c in cases]
    streams = [t.cuda.Stream() for _ in cases]
    out = [(t.empty_like(o), t.empty_like(lse)) for o, lse in want]
    for s in streams:
        sk.skgemm_reserve_ops(s)
    t.cuda.synchronize()
    for _ in range(10):
        for c, s, (o, lse) in zip(cases, streams, out):
            c.call(o, lse, stream=s)
    t.cuda.synchronize()
    for (o, lse), (a, b) in zip(out, want):
        assert t.equal(o, a) and t.equal(lse, b)


@pytest.mark.gpu
def test_cache_past_4_gib():
    """Offsets past 32 bits, in both strides' orders."""
    t = torch()
    c = Case([(1, 100), (50, 120)], 1, 4, 128, 16, "bf16", "token", seed=5)
    want = c.run()
    n = (5 << 30) // (16 * 128 * 2)
    big = [t.empty(n, 16, 1, 128, dtype=t.bfloat16, device=DEV) for _ in "kv"]
    far = n - c.n_pages
    for a, b in zip(big, (c.kc, c.vc)):
        a[far:] = b
    c.kc, c.vc = big
    c.n_pages = n
    c.table_d = t.where(c.table_d >= 0, c.table_d + far, c.table_d)
    got = c.run()
    assert all(t.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,max_q", [([(5, 60), (3, 9)], 2), ([(90, 200), (40, 40), (1, 7)], 33)])
def test_rows_past_max_q_are_left_out(seqs, max_q):
    """The rows before them sit where they would, the others are left as they were."""
    t = torch()
    c = Case(seqs, 2, 4, 128, 16, "bf16", "token", seed=9)
    want, wl = c.run()
    o, lse = c.run(max_q=max_q)
    for b, (n, _) in enumerate(seqs):
        a = int(c.starts[b])
        k = min(n, max_q)
        err = np.abs(f64(o[a : a + k]) - f64(want[a : a + k]))  # both within the bound of c.check, of the same value
        assert np.all(err <= 4 * O.EPS_BF16 * np.maximum(np.abs(f64(want[a : a + k])), np.abs(f64(c.values[1][b])).max()))
        assert np.allclose(lse[a : a + k].cpu(), wl[a : a + k].cpu(), rtol=0, atol=1e-4)
        assert (f64(o[a + k : a + n]) == 7.75).all() and (lse[a + k : a + n] == -55).all()


@pytest.mark.gpu
def test_attention_empty_calls():
    t = torch()
    x = t.zeros(0, 128, dtype=t.bfloat16, device=DEV)
    sk.skgemm_paged_attention(x, None, None, None, None, None, x, None, 0, 0, 0, 1, 1, 128, 0, 1, 0, 1.0)


A = 1 << 20  # an address; every call below is refused before any is used


def test_attention_refusals():
    f = sk.lib().skgemm_paged_attention

    def call(Q=A, K=A, V=A, table=A, lens=A, start=A, out=2 * A, lse=A, T=3, B=2, max_q=2, Hq=4, Hkv=2, D=128, n=9, page=16, most=4,
             scale=0.1, window=0, fmt=0, ks=1.0, vs=1.0, qs=1024, os=1024, ts=16, ps=8192, ss=512, hs=256):
        return f(Q, K, V, table, lens, start, out, lse, T, B, max_q, Hq, Hkv, D, n, page, most, scale, window, fmt, ks, vs, qs, os, ts, ps,
                 ss, hs, None)

    for name in ("T", "B", "max_q", "Hq", "Hkv", "n", "most", "window"):
        assert call(**{name: -1}) == sk.SKGEMM_EINVAL, name
    for name in ("Q", "K", "V", "table", "lens", "start", "out"):
        assert call(**{name: None}) == sk.SKGEMM_EINVAL, name
        assert call(**{name: A + 2}) == sk.SKGEMM_EALIGN, name
    assert call(lse=A + 2) == call(qs=1032) == call(os=1032) == call(ts=18) == call(ps=8200) == call(ss=520) == call(hs=264) == sk.SKGEMM_EALIGN
    for scale in (0.0, -1.0, float("nan"), float("inf"), 2.1e38, 1e-38):
        assert call(scale=scale) == sk.SKGEMM_EINVAL
    assert call(n=0) == call(page=0) == call(fmt=1) == call(ks=2.0) == call(fmt=2, vs=0.0) == call(fmt=2, scale=1e-20, ks=1e-20) == sk.SKGEMM_EINVAL
    for D in (32, 80, 96, 192, 512):
        assert call(D=D) == sk.SKGEMM_ESHAPE
    assert call(Hq=5) == call(Hkv=0) == call(page=12) == call(page=1 << 16) == call(Hq=4098) == call(B=1 << 21) == sk.SKGEMM_ESHAPE
    assert call(most=1 << 27) == call(T=1 << 21, Hq=2048, Hkv=1) == call(B=1 << 20, most=1 << 14) == sk.SKGEMM_ESHAPE
    assert call(out=A, os=2048) == call(os=512) == sk.SKGEMM_EINVAL
    for name in ("T", "B", "max_q", "Hq"):
        assert call(**{name: 0, "Q": None}) == sk.SKGEMM_OK


def test_attention_binding_refusals():
    t = torch()
    from tests.test_ops_binding import OnGpu

    def call(**kw):
        a = dict(Q=A, K=A, V=A, table=A, lens=A, start=A, O=2 * A, lse=A) | kw
        sk.skgemm_paged_attention(a["Q"], a["K"], a["V"], a["table"], a["lens"], a["start"], a["O"], a["lse"], 4, 2, 2, 2, 1, 64, 3, 16, 2,
                                  0.125, stream=0)

    z = lambda *s, ty=t.bfloat16: OnGpu(t.zeros(*s, dtype=ty))  # noqa: E731
    bad = [dict(Q=t.zeros(4, 128)), dict(Q=z(4, 128, ty=t.float16)), dict(Q=z(3, 128)), dict(O=z(4, 64)), dict(table=z(2, 2, ty=t.int64)),
           dict(lens=z(2, ty=t.int64)), dict(start=z(2, ty=t.int32)), dict(lse=z(4, 2)), dict(K=z(3, 16, 64)), dict(K=z(2, 16, 1, 64)),
           dict(K=z(3, 16, 1, 128)), dict(V=z(3, 16, 1, 64, ty=t.float16)), dict(K=z(3, 16, 1, 64), V=z(3, 1, 32, 64)),
           dict(K=z(3, 16, 1, 64, ty=t.float8_e4m3fn), V=z(3, 16, 1, 64))]
    for kw in bad:
        with pytest.raises(sk.SkgemmError) as e:
            call(**kw)
        assert e.value.code == sk.SKGEMM_EINVAL, kw
