"""The selection of a row's best tokens (logprobs.hip, block_top), on a host model.

A run of a row falls to 256 owners; each has a bound below its best key, a
threshold that k bounds reach picks the owners that are read again, and where
they hold more candidates than the buffer of 1024, the k-th key itself is
searched bit by bit. The ranking indexes the buffer by the number of candidates,
so that number has to be within it. The model follows the arithmetic of the
kernel and shows it for ordered values, equal ones and banned ones among them,
and that it fails for rows with NaN: the kernel selects nothing there.
"""

import numpy as np
import pytest

OWNERS, BUFFER = 256, 1024
U64 = np.uint64


def order_bits(v):
    b = (v.astype(np.float32) + np.float32(0)).view(np.uint32)
    return np.where(b & np.uint32(1 << 31), ~b, b | np.uint32(1 << 31))


def make_keys(v):
    index = ~np.arange(v.size, dtype=np.uint32)
    return (order_bits(v).astype(U64) << U64(32)) | index.astype(U64)


def owners_of(n):
    """The owner of each of n vectors, and the thread that reads it first."""
    rounds = -(-n // OWNERS)
    lg = 3 if rounds >= 8 else 2 if rounds >= 4 else 1 if rounds >= 2 else 0
    length = -(-rounds // (1 << lg))
    j = np.arange(n)
    seg, group = j // OWNERS // length, (j % OWNERS) >> lg
    return seg * (OWNERS >> lg) + group


def bounds_of(row, most, owner, per):
    """A bound below each owner's best key, as the pass over the data leaves it."""
    best = np.zeros(OWNERS, U64)
    for o in range(OWNERS):
        mine = np.flatnonzero(owner == o)
        if not mine.size:
            continue
        largest = np.fmax.reduce(np.where(np.isnan(most[mine]), -np.inf, most[mine]))
        held = mine[most[mine] == largest]
        # nothing but -inf: each thread keeps its first vector
        first = held[0] if held.size and largest > -np.inf else mine[0]
        low = ~np.uint32(first * per + per - 1)
        best[o] = (U64(order_bits(np.array([largest]))[0]) << U64(32)) | U64(low)
    return best


def threshold(best, k):
    value, index = (best >> U64(32)).astype(np.uint32), best.astype(np.uint32)
    valid = np.count_nonzero(value)
    if valid < k:
        return U64(0)
    slack = k // 2 + 8
    most, least = int(value.max()), int(value[value != 0].min())
    differ = most ^ least
    bit = 1 << (differ.bit_length() - 1) if differ else 0
    at = most & ~(2 * bit - 1) if bit else most
    reach, low_index = valid, 0
    while bit and reach > k + slack:
        n = np.count_nonzero(value >= at | bit)
        if n >= k:
            at, reach = at | bit, n
        bit >>= 1
    if reach > k + slack:
        low_index, low = 0xFFFFFFFF & ~((2 << 20) - 1), 1 << 20
        while low and reach > k + slack:
            n = np.count_nonzero((value > at) | ((value == at) & (index >= low_index | low)))
            if n >= k:
                low_index, reach = low_index | low, n
            low >>= 1
    return (U64(at) << U64(32)) | U64(low_index)


def select(row, per, k):
    """(candidates that the ranking is given, before any bound; the best k keys)."""
    n = row.size // per
    keys = make_keys(row).reshape(n, per)
    with np.errstate(invalid="ignore"):
        most = np.fmax.reduce(row.reshape(n, per), axis=1)
    owner = owners_of(n)
    best = bounds_of(row, most, owner, per)
    lowest = threshold(best, k)
    picked = (best != 0) & (best + U64(per - 1) >= lowest)
    live = picked[owner]
    reached = order_bits(most).astype(U64)  # a vector's largest, NaN passed over

    def candidates(c):
        at = live & (reached >= c >> U64(32))
        return keys[at][keys[at] >= c]

    got = candidates(lowest)
    if got.size > BUFFER:
        kth = 0
        for b in range(63, -1, -1):
            if candidates(U64(kth | 1 << b)).size >= k:
                kth |= 1 << b
        got = candidates(U64(kth))
    return got.size, np.sort(got)[::-1][:k]


def rows(n, rng):
    yield "normal", rng.standard_normal(n)
    yield "equal", np.full(n, 0.25)
    yield "banned but few", np.where(rng.random(n) < 0.999, -np.inf, rng.standard_normal(n))
    yield "half banned", np.where(rng.random(n) < 0.5, -np.inf, rng.standard_normal(n))
    yield "nothing but -inf", np.full(n, -np.inf)
    few = np.full(n, -1.0)
    few[(np.arange(n) // 8) % OWNERS < 3] = 5.0
    yield "few owners hold all", few
    yield "rounded", np.round(rng.standard_normal(n) * 4) / 4
    yield "ascending", np.linspace(-30, 30, n)


@pytest.mark.parametrize("per", [4, 8])
@pytest.mark.parametrize("n", [2048, 6144, 65536])
def test_ordered_values_stay_within_the_buffer(per, n):
    for k in (1, 20, 64):
        for what, row in rows(n, np.random.default_rng(n + k)):
            row = row.astype(np.float32)
            count, got = select(row, per, k)
            assert k <= count <= BUFFER, (what, k, count)
            assert np.array_equal(got, np.sort(make_keys(row))[::-1][:k]), (what, k)


def test_nan_rows_pass_the_buffer():
    """Why a run with a NaN is not selected from: a vector of NaN and -inf is left
    out until the search falls to -inf, and then all its NaN count at once: at
    least k owners of 64 vectors with four NaN each."""
    row = np.full(131072, -np.inf, np.float32)
    row[::2] = np.nan
    count, _ = select(row, 8, 64)
    assert count >= 64 * 64 * 4 > BUFFER
