"""skgemm_paged_attention with a window over tables whose old pages were given back
(the bounds of test_gpu_attention)."""

import pytest

from tests.gpu_util import log, torch
from tests.test_gpu_attention import Case

SINGLE = [(1, n) for n in range(90, 420, 11)]
CHUNKS = [(3, 310), (60, 700), (1, 333), (130, 500), (2, 1), (0, 200), (40, 45)]


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, None, 1 << 30])
@pytest.mark.parametrize("D,fmt", [(128, "bf16"), (64, "e4m3"), (256, "bf16")])
@pytest.mark.parametrize("page,order", [(1, "token"), (8, "head"), (16, "token"), (64, "head")])
@pytest.mark.parametrize("seqs,window", [(SINGLE, 100), (SINGLE, 1), ([(7, 5000)], 3001), ([(90, 900)], 257), ([(300, 6000)], 3100), (CHUNKS, 150)])
def test_window_over_released_pages(seqs, window, page, order, D, fmt, bad):
    """No page before the first token that a sequence's rows see is looked up: of few
    rows, of many, split and in one batch, the bits are those of the whole table."""
    t = torch()
    c = Case(seqs, 1, 4, D, page, fmt, order, pad=1, seed=window)
    log(f"attention window={window} over released pages, {seqs[-1]} D={D} {fmt} page={page} bad={bad}")
    want = c.run(window)
    for b, (n, L) in enumerate(seqs):
        c.table_d[b, : max(0, L - n + 1 - window) // page] = c.n_pages if bad is None else bad
    got = c.run(window)
    if page == 16:
        c.check(*got, window, rows=lambda n: sorted({0, n // 2, n - 1}))
    assert all(t.equal(a, b) for a, b in zip(got, want))
