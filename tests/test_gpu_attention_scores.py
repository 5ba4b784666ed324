"""skgemm_paged_attention where scores are of any size that FP32 holds."""

import numpy as np
import pytest

import split_reduction_amd as sk
from oracle import ops as O
from tests.gpu_util import DEV, log, torch


SIZES = [(1, 1), (1, 200), (1, 9000), (40, 300), (40, 9000)]


def check_equal_scores(n, L, D, scores, lower):
    """Every key has the score s, or every third one where `lower` is a factor that the
    others' is times. Equal scores have equal probabilities p <= 1, bf16's nearest to a
    power of two with an exponent that is off by less than half a step of s / log 2, and
    the others none (they are s / 16 lower, far below 2^-200). The values
    are small whole numbers: their sums are exact but for the p in front, so O is off by
    p's rounding, the sums' (L + 64 in FP32), the division (2) and the rounding to bf16. A score of -inf
    is no key: a row of nothing else has 0 and -inf.
    s is one product of bf16 numbers, times the scale and a factor (3 roundings); lse
    turns it back (2), adding log L (1)."""
    t = torch()
    G, page = 2, 64
    pages = -(-L // page)
    rng = np.random.default_rng(L)
    kc = t.zeros(pages, page, 1, D, dtype=t.bfloat16, device=DEV)
    kc[..., 3] = -(2.0**60)
    top = np.ones(pages * page, bool)
    if lower:
        top[np.arange(pages * page) % 3 != 0] = False
        kc.view(-1, D)[t.from_numpy(~top).to(DEV), 3] *= lower
    values = rng.integers(-8, 9, (L, D)).astype(np.float64)
    vc = t.zeros(pages * page, D)
    vc[:L] = t.from_numpy(values).float()
    vc = vc.to(t.bfloat16).view(pages, page, 1, D).to(DEV)
    table = t.arange(pages, dtype=t.int32, device=DEV).view(1, -1)
    lens, start = t.tensor([L], dtype=t.int32, device=DEV), t.tensor([0, n], dtype=t.int32, device=DEV)
    for s in scores:
        x = t.tensor(-s / 2.0**60 * 8 if np.isfinite(s) else 1.0).to(t.bfloat16)  # scale 1 / 8
        s = -float(x) * 2.0**60 / 8 if np.isfinite(s) else s
        q = t.zeros(n, G, D, dtype=t.bfloat16, device=DEV)
        q[..., 3] = x
        kc[..., 3] *= float("inf") if np.isinf(s) else 1.0
        o = t.full((n, G, D), 7.0, dtype=t.bfloat16, device=DEV)
        lse = t.full((n, G), 7.0, device=DEV)
        sk.skgemm_paged_attention(q, kc, vc, table, lens, start, o, lse, n, 1, n, G, 1, D, pages, page, pages, 0.125)
        t.cuda.synchronize()
        got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
        if np.isinf(s):
            assert (got == 0).all() and np.isneginf(gl).all()
            continue
        for i in range(n):
            seen = values[: L - n + i + 1][top[: L - n + i + 1]]
            ref, size = seen.mean(0), np.abs(seen).mean(0)
            assert np.all(np.abs(got[i] - ref) <= np.abs(ref) * O.EPS_BF16 * 2 + size * (O.EPS_BF16 + (L + 67) * O.EPS_F32)), (s, i)
        assert np.all(np.abs(gl - s) <= 6 * O.EPS_F32 * abs(s) + np.log(L)), s


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,L", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(n, L, D, sign):
    log(f"attention of large scores n={n} L={L} D={D} sign={sign}")
    scores = [sign * s for s in (1e7, 3.3e9, 4.7e9, 1.1e10, 1.3e13, 2.9e17, 7e20, 1e25, 5.7e29)]
    check_equal_scores(n, L, D, scores, None)
    check_equal_scores(n, L, D, scores, 1 - sign * 2.0**-4)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,L", SIZES)
def test_scores_near_the_lowest(n, L, D):
    log(f"attention near the lowest score n={n} L={L} D={D}")
    check_equal_scores(n, L, D, (-0.5e30, -0.75e30, -0.98e30, -1.02e30, -3e30, -1e36, -3e37, -np.inf), None)
