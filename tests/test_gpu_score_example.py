"""examples/score_tokens.py: the operators one after another, against fp64 from
the codes that the norm made. The logits round three times (see test_gpu_i8), so
z is within 3 * 2^-24 |z|; the log probabilities add their own bounds, here taken
together: 2^-24 * (8 max |z| + the sums' additions and joins (V / 256 + 64) + 16)."""

import importlib.util
import os

import numpy as np
import pytest

from oracle import ops as O
from tests.conftest import ROOT
from tests.gpu_util import DEV, torch


def example():
    spec = importlib.util.spec_from_file_location("score_tokens", os.path.join(ROOT, "examples", "score_tokens.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(1, 256, 1000), (9, 1024, 4099), (150, 512, 2050)])
def test_score_tokens(T, H, V):
    t = torch()
    t.manual_seed(T)
    bf16 = lambda *s: t.randn(*s, device=DEV).to(t.bfloat16)  # noqa: E731
    head = example().Head(1 + 0.1 * bf16(H), 0.05 * bf16(V, H))
    head.reserve(T + 3, 4)  # more rows than used
    x, r, tokens = bf16(T, H), bf16(T, H), t.randint(0, V, (T,), device=DEV)
    temperature = 0.5
    logprob, entropy, top, ids = head.score(x, r, tokens, temperature)
    f64 = lambda a: a.double().cpu().numpy()  # noqa: E731
    _, want = O.rmsnorm_ref(f64(x), f64(r), f64(head.norm_weight), head.eps)
    codes = head.q[:T].cpu().numpy()
    assert np.all(np.abs(codes * f64(head.q_scale)[:T, None] - want) <= O.row_scale(want, "i8")[:, None] * 0.5001)
    _, z = O.i8_ref(codes, head.q_scale[:T].cpu().numpy(), head.codes.cpu().numpy(), head.scale.cpu().numpy())
    ref = O.logprobs_ref(z, tokens.cpu().numpy(), 4, 1 / temperature)
    tol = O.EPS_F32 * (8 * np.abs(z).max() / temperature + V / 256 + 80)
    assert np.abs(f64(logprob) - ref["logprob"]).max() <= tol
    assert np.abs(f64(top) - ref["top"]).max() <= tol
    # the entropy weighs each term's error by its distance from the largest
    assert np.abs(f64(entropy) - ref["entropy"]).max() <= tol * (1 + np.log(V))
    d = f64(head.grad(tokens, t.ones(T, device=DEV), t.zeros(T, device=DEV), temperature))
    want, _, _ = O.logprobs_grad_ref(z, tokens.cpu().numpy(), ref["lse"], ref["entropy"], np.ones(T), np.zeros(T), 1 / temperature)
    assert np.abs(d - want).max() <= tol / temperature
    # replays of the captured calls give the eager bits
    eager = [a.clone() for a in head.score(x, r, tokens, temperature)]
    g = t.cuda.CUDAGraph()
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        example().sk.skgemm_reserve_ops(s)
    t.cuda.synchronize()
    with t.cuda.graph(g, stream=s):
        got = head.score(x, r, tokens, temperature)
    for _ in range(3):
        for a in got:
            a.zero_()
        g.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(got, eager))


@pytest.mark.gpu
def test_example_runs(capsys):
    example().main(3, 256, 1001)
    assert "row 2: token" in capsys.readouterr().out
