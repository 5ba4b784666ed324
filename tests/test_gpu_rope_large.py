"""Calls of skgemm_rope and skgemm_rope_append that move more than the last cache
holds give the bits of the same tokens in small calls (which test_gpu_rope checks)."""

import pytest

import split_reduction_amd as sk
from tests.gpu_util import DEV, log, torch


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,norm,layout", [(8200, 64, True, "half"), (8200, 64, False, "interleaved"), (110000, 5, True, "half")])
def test_many_tokens(T, H, norm, layout):
    t = torch()
    D = 128
    log(f"rope T={T} H={H} {layout} norm={norm}")
    t.manual_seed(T)
    x = t.randn(T, H * D, device=DEV).to(t.bfloat16)
    g = t.randn(D, device=DEV).to(t.bfloat16) if norm else None
    freq, pos = t.rand(D // 2, device=DEV), t.randint(0, 100000, (T,), device=DEV)
    y = t.empty_like(x)
    sk.skgemm_rope(x, g, freq, pos, y, T, H, D, D, layout)
    part = t.empty_like(x[:100])
    for a in [*range(0, T - 100, T // 9), T - 100]:
        sk.skgemm_rope(x[a : a + 100], g, freq, pos[a : a + 100], part, 100, H, D, D, layout)
        t.cuda.synchronize()
        assert t.equal(part, y[a : a + 100]), a


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,Hq,Hkv,order", [(8200, 56, 8, "head"), (40000, 8, 8, "token")])
def test_many_appends(T, Hq, Hkv, order, fmt):
    t = torch()
    D, page = 128, 16
    log(f"append T={T} {Hq}+{Hkv} {order} {fmt}")
    t.manual_seed(T)
    rows = t.randn(T, (Hq + 2 * Hkv) * D, device=DEV).to(t.bfloat16)
    gq, gk = (t.randn(D, device=DEV).to(t.bfloat16) for _ in "qk")
    freq, pos = t.rand(D // 2, device=DEV), t.randint(0, 100000, (T,), device=DEV)
    pages = -(-T // page) + 1
    slots = t.randperm(pages * page, device=DEV)[:T]
    kind, ks, vs = (t.float8_e4m3fn, 0.3, 0.07) if fmt == "e4m3" else (t.bfloat16, 1.0, 1.0)
    shape = (pages, page, Hkv, D) if order == "token" else (pages, Hkv, page, D)

    def run(a, b):
        n = b - a
        kc, vc = (t.zeros(shape, dtype=kind, device=DEV) for _ in "kv")
        if order == "head":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        q, k, v = rows[a:b].split((Hq * D, Hkv * D, Hkv * D), 1)
        out = t.empty(n, Hq * D, dtype=t.bfloat16, device=DEV)
        sk.skgemm_rope_append(q, k, v, gq, gk, freq, pos[a:b], slots[a:b], out, kc, vc, n, Hq, Hkv, D, pages, page, D, k_scale=ks, v_scale=vs)
        t.cuda.synchronize()
        at = slots[a:b]
        return out, *(c.view(t.uint8)[at // page, at % page] for c in (kc, vc))

    whole = run(0, T)
    for a in [*range(0, T - 100, T // 5), T - 100]:
        assert all(t.equal(p, w[a : a + 100]) for p, w in zip(run(a, a + 100), whole)), a
