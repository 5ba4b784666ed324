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


@pytest.mark.gpu
@pytest.mark.parametrize("D,fmt", [(128, "bf16"), (128, "e4m3"), (64, "bf16"), (64, "e4m3"), (256, "bf16"), (256, "e4m3")])
def test_one_chunk_with_split_keys(D, fmt):
    """Tiles of 256 rows where there is such a form, and each one's keys over workgroups."""
    c = Case([(300, 6000)], 2, 4, D, 32, fmt, "head", seed=D)
    log(f"attention chunk with split keys D={D} {fmt}")
    c.check(*c.run(), rows=lambda n: [0, 63, 64, 127, 200, n - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("beside", [[], [(40, 50), (1, 3)]])
@pytest.mark.parametrize("D,fmt", [(128, "bf16"), (128, "e4m3"), (64, "bf16"), (64, "e4m3"), (256, "bf16"), (256, "e4m3")])
def test_many_parts_of_a_head(D, fmt, beside):
    """32 rows over 40000 keys of one head: 79 workgroups' parts, past the 32 or 64 whose
    maxima a join takes at once."""
    c = Case([(4, 40000), *beside], 1, 8, D, 64, fmt, "head", seed=D + len(beside))
    log(f"attention many parts D={D} {fmt} beside {beside}")
    c.check(*c.run(), rows=ENDS)


@pytest.mark.gpu
@pytest.mark.parametrize("D,fmt", [(64, "bf16"), (128, "e4m3")])
def test_tiles_past_the_counters(D, fmt):
    """Splits would need more counters than there are: none, whatever the keys."""
    seqs = [(33 + b % 5, 40 + b % 7) if b % 3 else (1 + b % 2, 30) for b in range(299)] + [(40, 1500)]
    c = Case(seqs, 32, 1, D, 16, fmt, "token", seed=D)
    log(f"attention tiles past the counters D={D} {fmt}")
    c.check(*c.run(), rows=lambda n: [n - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("most", [1, 50])
@pytest.mark.parametrize("D,fmt", [(128, "bf16"), (64, "e4m3")])
def test_thousands_of_sequences(D, fmt, most):
    """Each workgroup looks at 64 at a time; of the second kind some are of many rows."""
    seqs = [(most if b % 50 == 7 else b % 3 if most > 1 else 1, 60 + b % 41) for b in range(2100)]
    c = Case(seqs, 1, 2, D, 16, fmt, "head", pad=1, seed=most)
    log(f"attention of {len(seqs)} sequences D={D} {fmt}")
    c.check(*c.run(), rows=lambda n: [n - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["token", "head"])
def test_caches_past_4_gib_of_two_heads(order):
    """Offsets of pages past 32 bits, with a page's tokens and with its heads first."""
    t = torch()
    c = Case([(1, 100), (50, 120)], 2, 4, 128, 16, "bf16", order, seed=5)
    want = c.run()
    n = (5 << 30) // (16 * 2 * 128 * 2)
    far, big = n - c.n_pages, []
    for a in c.mem:
        b = t.empty(n, *a.shape[1:], dtype=t.bfloat16, device=DEV)
        b[far:] = a
        big.append(b)
    c.kc, c.vc = big if order == "token" else [b.transpose(1, 2) for b in big]
    c.n_pages = n
    c.table_d = t.where(c.table_d >= 0, c.table_d + far, c.table_d)
    got = c.run()
    assert all(t.equal(a, b) for a, b in zip(got, want))
