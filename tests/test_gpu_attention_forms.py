"""skgemm_paged_attention in each of the forms that a call may take: by rows of a key
head (up to 32 or more), sequences, keys and heads (the bounds of test_gpu_attention)."""

import pytest

from tests.gpu_util import DEV, log, torch
from tests.test_gpu_attention import Case

ENDS = lambda n: sorted({0, n // 3, n - 1})  # noqa: E731


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,L,Hkv,G", [(3001, 3001, 9, 8), (2900, 3050, 2, 40), (7000, 7000, 4, 8)])
def test_long_prompts(n, L, Hkv, G, fmt):
    """Tiles of 256 rows that outnumber the CUs three times, keys not split."""
    c = Case([(n, L)], Hkv, G, 128, 32, fmt, "head", pad=1, seed=n)
    log(f"attention long prompt n={n} L={L} {Hkv} key heads of {G} {fmt}")
    c.check(*c.run(), rows=lambda n: [0, 1, 31, n // 2, n - 1])
