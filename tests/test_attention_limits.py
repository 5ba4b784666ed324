"""Sizes of skgemm_paged_attention past what one launch takes."""

import split_reduction_amd as sk

A = 1 << 20  # an address; every call below is refused before any is used


def test_more_workgroups_than_a_launch_takes():
    def call(T=1 << 21, B=1 << 20, max_q=40, Hq=64, Hkv=16):
        return sk.lib().skgemm_paged_attention(A, A, A, A, A, A, 2 * A, A, T, B, max_q, Hq, Hkv, 128, 9, 16, 4, 0.1, 0, 0, 1.0, 1.0, Hq * 256,
                                               Hq * 256, 16, Hkv * 4096, Hkv * 256, 256, None)

    assert call() == sk.SKGEMM_ESHAPE
    assert call(B=(1 << 20) - 65536 - 32) == sk.SKGEMM_ESHAPE  # the first that is too many: tiles of T / 32 + B, 16 heads
    assert call(B=1 << 13, T=1 << 21, Hq=2048, Hkv=512, max_q=2000) == sk.SKGEMM_ESHAPE
    assert call(B=1 << 18, T=1 << 21, Hq=64 * 16, Hkv=64, max_q=3) == sk.SKGEMM_ESHAPE  # one tile a sequence
