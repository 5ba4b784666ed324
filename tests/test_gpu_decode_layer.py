"""examples/decode_layer.py: products, head norm and rotation, cache and attention one
after another, each step against fp64 from what the step before left on the GPU (the
bounds of test_gpu_rope and test_gpu_attention; the products' as everywhere)."""

import importlib.util
import os

import numpy as np
import pytest

from oracle import formats as F
from oracle import gemm as G
from oracle import ops as O
from tests.conftest import ROOT
from tests.gpu_util import assert_parity, bf16_bits, log, torch
from tests.test_gpu_rope import close, close_codes, f64

E = O.EPS_F32


def example():
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def check_step(m, block, cache, x, counts):
    """One run of the block, and every call's outputs from its inputs."""
    t = torch()
    H, Hq, Hkv, D, T = block.H, block.Hq, block.Hkv, block.D, sum(counts)
    pos, slots, length, start = cache.take(counts)
    y = block.run(x, cache, pos, slots, length, start, max(counts))
    t.cuda.synchronize()
    bits = lambda a: bf16_bits(a[:T])  # noqa: E731
    assert_parity(bits(block.rows), G.gemm_bf16_ref(bits(block.h), bf16_bits(block.qkv)), H, "queries, keys, values")
    rows = f64(block.rows[:T]).reshape(T, Hq + 2 * Hkv, D)
    freq, p = block.freq.cpu().numpy(), pos.cpu().numpy()
    ref, size = O.rope_ref(rows[:, :Hq], f64(block.q_norm), freq, p, D, "half", block.eps)
    q = f64(block.q[:T]).reshape(T, Hq, D)
    close(q, ref, size, "queries")
    ref, size = O.rope_ref(rows[:, Hq : Hq + Hkv], f64(block.k_norm), freq, p, D, "half", block.eps)
    at = slots.cpu().numpy()
    v = rows[:, Hq + Hkv :]
    if cache.k.element_size() == 1:
        code = lambda c: c.view(t.uint8).contiguous().cpu().numpy().reshape(-1, Hkv, D)  # noqa: E731
        close_codes(code(cache.k)[at], ref, size, cache.k_scale, "keys")
        close_codes(code(cache.v)[at], v, np.abs(v), cache.v_scale, "values")
        held = [F.e4m3_value(code(c)) * s for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    else:
        held = [f64(c).reshape(-1, Hkv, D) for c in (cache.k, cache.v)]
        close(held[0][at], ref, size, "keys")
        assert np.array_equal(held[1][at], v)
    o = f64(block.o[:T]).reshape(T, Hq, D)
    table, first = cache.table.cpu().numpy(), 0
    for b, n in enumerate(counts):
        L = cache.length[b]
        mine = table[b, np.arange(L) // m.PAGE] * m.PAGE + np.arange(L) % m.PAGE
        ref, _, A, S = O.attention_ref(q[first : first + n], held[0][mine], held[1][mine], D**-0.5)
        soft = (2 * S * (D + 4) + 2 * S + 2 * L + 133) * E + O.EPS_BF16
        tol = A * soft[:, :, None] * (1 + O.EPS_BF16) + O.EPS_BF16 * np.abs(ref) + 2.0**-133
        assert np.all(np.abs(o[first : first + n] - ref) <= tol), (b, n, L)
        first += n
    assert_parity(bits(block.y), G.gemm_bf16_ref(bits(block.o), bf16_bits(block.out)), Hq * D, "output")
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,codes", [(16, 2, 128, False), (8, 8, 64, False), (4, 2, 256, True), (16, 2, 128, True)])
def test_prompts_chunks_and_tokens(Hq, Hkv, D, codes):
    t = torch()
    m = example()
    t.manual_seed(Hq)
    H, B = 512, 3
    log(f"decode layer Hq={Hq} Hkv={Hkv} D={D} codes={codes}")
    block = m.Block(H, Hq, Hkv, D, 128)
    kind = dict(dtype=t.float8_e4m3fn, k_scale=0.03, v_scale=0.02) if codes else {}
    cache = m.Cache(64, Hkv, D, B, 200, **kind)
    x = lambda n: t.randn(n, H, device="cuda").to(t.bfloat16)  # noqa: E731
    for counts in ([37, 5, 60], [1, 0, 1], [1, 40, 1], [1, 1, 1], [0, 3, 0], [1, 1, 1]):
        check_step(m, block, cache, x(sum(counts)), counts)


@pytest.mark.gpu
def test_token_steps_captured():
    """A step of single tokens as a graph, replayed with other lengths and pages, gives
    the eager bits."""
    t = torch()
    m = example()
    t.manual_seed(7)
    H, Hq, Hkv, D, B = 512, 16, 2, 128, 4
    block = m.Block(H, Hq, Hkv, D, 256)
    caches = [m.Cache(80, Hkv, D, B, 300) for _ in range(2)]
    first = [50, 3, 120, 17]
    x = t.randn(sum(first), H, device="cuda").to(t.bfloat16)
    for c in caches:
        block.run(x, c, *c.take(first), max(first))
    steps = [t.randn(B, H, device="cuda").to(t.bfloat16) for _ in range(4)]
    eager = [block.run(s, caches[0], *caches[0].take([1] * B), 1).clone() for s in steps]
    t.cuda.synchronize()
    xs = steps[0].clone()
    held = [a.clone() for a in caches[1].take([1] * B)]
    stream = t.cuda.Stream()
    with t.cuda.stream(stream):
        m.sk.skgemm_reserve_ops()
        m.sk.skgemm_reserve(B, (Hq + 2 * Hkv) * D, 4)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=stream):
        y = block.run(xs, caches[1], *held, 1)
    for i, s in enumerate(steps):
        if i:
            xs.copy_(s)
            for a, b in zip(held, caches[1].take([1] * B)):
                a.copy_(b)
        g.replay()
        t.cuda.synchronize()
        assert t.equal(y, eager[i]), i
    del g


@pytest.mark.gpu
def test_example_runs(capsys):
    example().main(3)
    assert "after 3 tokens more each: lengths [40, 203, 4]" in capsys.readouterr().out
