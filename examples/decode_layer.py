"""The attention block of a decoding layer, in five calls.

The norm, the product for queries, keys and values, the norm of the heads with the
rotation on the way into a paged cache, the attention over that cache, and the output
product. A prompt, a chunk of it and single tokens go the same way. Weights are
random: the example shows the calls and their buffers.

    python examples/decode_layer.py [tokens to generate]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import split_reduction_amd as sk  # noqa: E402

PAGE = 16


class Cache:
    """Pages of keys and values [pages, PAGE, Hkv, D], a head's tokens of a page next to
    each other, and each sequence's pages, handed out in turn."""

    def __init__(self, pages, Hkv, D, B, max_len, dtype=torch.bfloat16, k_scale=1.0, v_scale=1.0):
        new = lambda: torch.zeros(pages, Hkv, PAGE, D, dtype=dtype, device="cuda").transpose(1, 2)  # noqa: E731
        self.k, self.v = new(), new()
        self.k_scale, self.v_scale = k_scale, v_scale
        self.max_pages = -(-max_len // PAGE)
        self.table = torch.full((B, self.max_pages), -1, dtype=torch.int32, device="cuda")
        self.length = [0] * B
        self.free = list(range(pages))

    def take(self, counts):
        """Room for counts[b] new tokens of each sequence: their positions and slots, the
        lengths with them and where each sequence's rows start."""
        positions, slots, start = [], [], [0]
        for b, n in enumerate(counts):
            old, new = self.length[b], self.length[b] + n
            for page in range(-(-old // PAGE), -(-new // PAGE)):
                self.table[b, page] = self.free.pop()
            pages = self.table[b].tolist()
            positions += range(old, new)
            slots += [pages[p // PAGE] * PAGE + p % PAGE for p in range(old, new)]
            self.length[b] = new
            start.append(start[-1] + n)
        on_gpu = lambda a, t: torch.tensor(a, dtype=t, device="cuda")  # noqa: E731
        return (on_gpu(positions, torch.int64), on_gpu(slots, torch.int64), on_gpu(self.length, torch.int32),
                on_gpu(start, torch.int32))


class Block:
    """Norm, queries, keys and values, attention and output product of H features."""

    def __init__(self, H, Hq, Hkv, D, max_rows, base=10000.0, eps=1e-6):
        self.H, self.Hq, self.Hkv, self.D, self.eps = H, Hq, Hkv, D, eps
        w = lambda n, k: (torch.randn(n, k, device="cuda") * k**-0.5).to(torch.bfloat16)  # noqa: E731
        self.qkv, self.out = w((Hq + 2 * Hkv) * D, H), w(H, Hq * D)
        gain = lambda n: (1 + 0.1 * torch.randn(n, device="cuda")).to(torch.bfloat16)  # noqa: E731
        self.norm, self.q_norm, self.k_norm = gain(H), gain(D), gain(D)
        self.freq = torch.pow(base, -torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D).float()
        new = lambda n: torch.empty(max_rows, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.h, self.rows, self.q, self.o, self.y = new(H), new((Hq + 2 * Hkv) * D), new(Hq * D), new(Hq * D), new(H)
        sk.skgemm_reserve_ops()

    def run(self, x, cache, positions, slots, length, start, max_new):
        """x [T, H]: the rows of all sequences' new tokens, max_new of one at most."""
        T, Hq, Hkv, D = x.shape[0], self.Hq, self.Hkv, self.D
        sk.skgemm_rmsnorm(x, None, self.norm, None, self.h, None, T, self.H, self.eps)
        sk.skgemm_bf16(self.qkv, self.h, self.rows, T, (Hq + 2 * Hkv) * D, self.H, 4)
        q, k, v = self.rows[:T].split((Hq * D, Hkv * D, Hkv * D), 1)
        sk.skgemm_rope_append(q, k, v, self.q_norm, self.k_norm, self.freq, positions, slots, self.q, cache.k, cache.v, T, Hq, Hkv, D,
                              cache.k.shape[0], PAGE, D, "half", self.eps, k_scale=cache.k_scale, v_scale=cache.v_scale)
        sk.skgemm_paged_attention(self.q, cache.k, cache.v, cache.table, length, start, self.o, None, T, len(cache.length), max_new, Hq,
                                  Hkv, D, cache.k.shape[0], PAGE, cache.max_pages, D**-0.5, k_scale=cache.k_scale, v_scale=cache.v_scale)
        sk.skgemm_bf16(self.out, self.o, self.y, T, self.H, Hq * D, 4)
        return self.y[:T]


def main(steps=8):
    torch.manual_seed(0)
    H, Hq, Hkv, D = 2048, 16, 2, 128
    prompts = [37, 200, 1]
    block = Block(H, Hq, Hkv, D, sum(prompts))
    cache = Cache(64, Hkv, D, len(prompts), 300)
    x = torch.randn(sum(prompts), H, device="cuda").to(torch.bfloat16)
    y = block.run(x, cache, *cache.take(prompts), max(prompts))
    print(f"prompts of {prompts}: outputs of rms {y.float().pow(2).mean().sqrt().item():.3f}")
    for _ in range(steps):
        last = torch.cumsum(torch.tensor([1] * len(prompts)), 0) - 1 if y.shape[0] == len(prompts) else torch.cumsum(torch.tensor(prompts), 0) - 1
        x = y[last.cuda()].contiguous()
        y = block.run(x, cache, *cache.take([1] * len(prompts)), 1)
    print(f"after {steps} tokens more each: lengths {cache.length}, outputs of rms {y.float().pow(2).mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
