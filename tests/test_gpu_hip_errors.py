"""HIP keeps the last error of a thread until somebody asks for it. A call does not
report one that its caller left, and leaves none of its own behind."""

import ctypes

import pytest

import split_reduction_amd as sk
from tests.gpu_util import DEV, torch


def hip(name, *args):
    f = getattr(sk.lib(), name)  # of the runtime that the library is bound to
    f.restype = ctypes.c_int
    return f(*args)


@pytest.mark.gpu
def test_errors_of_the_caller_are_not_reported():
    t = torch()
    bf16 = lambda *s: t.randn(*s, device=DEV).to(t.bfloat16)  # noqa: E731
    x, w, c, z = bf16(8, 1024), bf16(512, 1024), bf16(8, 512), t.randn(8, 4000, device=DEV)
    q, f = t.zeros(512, 1024, dtype=t.int8, device=DEV), t.zeros(512, device=DEV)
    tok = t.zeros(8, dtype=t.int64, device=DEV)
    words = t.zeros(4096, dtype=t.int32, device=DEV)
    big, x100, c100 = t.empty(512, 512, device=DEV), bf16(100, 1024), bf16(100, 512)
    t.cuda.synchronize()
    calls = [
        lambda: sk.skgemm_rmsnorm(x, None, None, None, q[:8], f, 8, 1024, 1e-6, "i8"),
        lambda: sk.skgemm_i8(q, f, q[:8], f, c, 8, 512, 1024),
        lambda: sk.skgemm_i8(q, f, q, f, big, 512, 512, 1024),
        lambda: sk.skgemm_logprobs(z, tok, f, f, f, None, None, 8, 4000),
        lambda: sk.skgemm_logprobs_grad(z, tok, f, f, f, f, z, 8, 4000),
        lambda: sk.skgemm_bf16(w, x, c, 8, 512, 1024, 4),
        lambda: sk.skgemm_bf16(w, x100, c100, 100, 512, 1024, 2),
        lambda: sk.skgemm_read_probe(w, 4096, words),
    ]
    for kind in (0, 1):  # the GEMM's other kernels (the calls above take the cluster and the wide one)
        def pinned(kind=kind):
            sk.skgemm_set_override("kind", kind)
            try:
                sk.skgemm_bf16(w, x, c, 8, 512, 1024, 4)
            finally:
                sk.clear_overrides()
        calls.append(pinned)
    for call in calls:
        call()  # its workspace exists from here on
    t.cuda.synchronize()
    for i, call in enumerate(calls):
        assert hip("hipSetDevice", 4096) != 0
        call()
        assert hip("hipGetLastError") != 0, i  # the caller's error is still the caller's
    t.cuda.synchronize()


@pytest.mark.gpu
def test_a_failed_reserve_leaves_no_error():
    t = torch()
    t.zeros(1, device=DEV)
    hip("hipGetLastError")
    with pytest.raises(sk.SkgemmError) as e:
        sk.skgemm_reserve_batched(128, 1 << 18, 8, 4096)  # 4.4 TB
    assert e.value.code == sk.SKGEMM_ENOMEM
    assert hip("hipGetLastError") == 0
