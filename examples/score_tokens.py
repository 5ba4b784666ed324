"""Scoring tokens with a quantised language-model head, in four calls.

The last residual is added and normed into 8-bit codes, the codes are multiplied
with the head's 8-bit weights, and the logits give the log probability of each
row's token, the entropy and the best alternatives; a gradient to the logits
follows for whoever trains on them. Weights are random: the example shows the
calls and their buffers.

    python examples/score_tokens.py [rows]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import split_reduction_amd as sk  # noqa: E402


class Head:
    """The final norm and the output projection of a model, weights held as
    int8 codes with one scale for each of the V tokens."""

    def __init__(self, norm_weight, weight, eps=1e-6):
        top = weight.float().abs().amax(1, keepdim=True)
        self.codes = torch.round(weight.float() * (127 / top)).to(torch.int8)
        self.scale = (top / 127)[:, 0].contiguous()
        self.norm_weight, self.eps = norm_weight, eps
        self.V, self.H = weight.shape

    def reserve(self, max_rows, k):
        """Buffers for up to max_rows rows and k alternatives, and the stream's
        workspace: score() then allocates nothing and may be captured."""
        dev = self.codes.device
        new = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=dev)  # noqa: E731
        self.q, self.q_scale = new(max_rows, self.H, t=torch.int8), new(max_rows)
        self.residual = new(max_rows, self.H, t=torch.bfloat16)
        self.logits = new(max_rows, self.V)
        self.logprob, self.entropy, self.lse = new(max_rows), new(max_rows), new(max_rows)
        self.top, self.ids = new(max_rows, k), new(max_rows, k, t=torch.int64)
        self.k = k
        sk.skgemm_reserve_ops()

    def score(self, x, residual, tokens, temperature=1.0):
        """Row t of x + residual through the head, scored at tokens[t]."""
        T = x.shape[0]
        sk.skgemm_rmsnorm(x, residual, self.norm_weight, self.residual, self.q, self.q_scale, T, self.H, self.eps, "i8")
        sk.skgemm_i8(self.codes, self.scale, self.q, self.q_scale, self.logits, T, self.V, self.H)
        sk.skgemm_logprobs(self.logits, tokens, self.logprob, self.entropy, self.lse, self.top, self.ids, T, self.V,
                           self.k, 1 / temperature)
        return self.logprob[:T], self.entropy[:T], self.top[:T], self.ids[:T]

    def grad(self, tokens, g_logprob, g_entropy, temperature=1.0):
        """The gradient of sum(g_logprob * logprob) + sum(g_entropy * entropy) of
        the last score() to its logits, written over them."""
        T = tokens.shape[0]
        sk.skgemm_logprobs_grad(self.logits, tokens, self.lse, self.entropy, g_logprob, g_entropy, self.logits, T, self.V,
                                1 / temperature)
        return self.logits[:T]


def main(rows=16, H=1024, V=32001):
    torch.manual_seed(0)
    bf16 = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    head = Head(1 + 0.1 * bf16(H), 0.05 * bf16(V, H))
    head.reserve(rows, 5)
    tokens = torch.randint(0, V, (rows,), device="cuda")
    logprob, entropy, top, ids = head.score(bf16(rows, H), bf16(rows, H), tokens)
    for t in range(min(rows, 4)):
        best = ", ".join(f"{i} ({v:.2f})" for i, v in zip(ids[t].tolist(), top[t].tolist()))
        print(f"row {t}: token {tokens[t].item()} {logprob[t].item():.3f}, entropy {entropy[t].item():.3f}, best {best}")
    d = head.grad(tokens, torch.ones(rows, device="cuda"), torch.zeros(rows, device="cuda"))
    print(f"gradient of the summed log probabilities: row sums at most {d.sum(1).abs().max().item():.1e}")


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
