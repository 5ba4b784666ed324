"""The operators between a layer's first and last product, as they are measured.

Three operators: the norm of each head with the rotation by position (``rope``), the same for queries and keys
on the way of keys and values into a paged cache (``append``), and the attention of new tokens over that cache
(``attn``). ``step`` is an append and the attention that reads it, as a decoding layer runs them.

With ``own`` false a pass is the plain form, elementary torch operations in 32 bits (64 for the angles), rounded
once at the end; with ``own`` true it is the call a program makes of ``split_reduction_amd``.
"""

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BASE = 10000.0
K_SCALE, V_SCALE = 0.125, 0.03125  # of a cache of E4M3 codes
KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ---- the cases ---------------------------------------------------------------------------------------------
#
# T tokens, Hq and Hkv heads of queries and of keys, D values a head of which `rot` are rotated. An attention has
# B sequences of up to n new tokens and up to L tokens in all; where "mix" is "even" all have just these. "order"
# says which index of a cache's page comes first in memory: its tokens or its heads.


def listed():
    return [
        # the heads of one new token: launch latency
        {"name": "rope_t1_h16_d128", "op": "rope", "T": 1, "H": 16, "D": 128, "rot": 128, "style": "half", "norm": True, "far": 4096},
        # a long prompt's queries, a part of each head rotated, positions far out: memory traffic
        {"name": "rope_t8192_h64_d128", "op": "rope", "T": 8192, "H": 64, "D": 128, "rot": 64, "style": "interleaved", "norm": False,
         "far": 1000000},
        # one decode step of a ragged batch into a cache
        {"name": "append_t67_h16_2_d128", "op": "append", "T": 67, "Hq": 16, "Hkv": 2, "D": 128, "rot": 128, "style": "half", "norm": True,
         "far": 32768, "page": 16, "kind": "bf16", "order": "token"},
        # a prompt's rows into a cache of 8 bits: memory traffic
        {"name": "append_t8192_h64_8_d128", "op": "append", "T": 8192, "Hq": 64, "Hkv": 8, "D": 128, "rot": 128, "style": "half",
         "norm": True, "far": 131072, "page": 64, "kind": "e4m3", "order": "head"},
        # one token of one short conversation: launch latency
        {"name": "attn_b1_n1_l257_d128", "op": "attn", "B": 1, "n": 1, "L": 257, "mix": "even", "pad": 0, "Hq": 16, "Hkv": 2, "D": 128,
         "page": 16, "kind": "bf16", "order": "token", "window": 0},
        # a decode batch of conversations of all lengths: the cache's traffic
        {"name": "attn_b64_n1_l16000_d128", "op": "attn", "B": 64, "n": 1, "L": 16000, "mix": "ragged", "pad": 0, "Hq": 64, "Hkv": 8,
         "D": 128, "page": 16, "kind": "bf16", "order": "head", "window": 0},
        # one token over a very long text in 8 bits: few rows, a long axis
        {"name": "attn_b1_n1_l131072_d128", "op": "attn", "B": 1, "n": 1, "L": 131072, "mix": "even", "pad": 0, "Hq": 64, "Hkv": 8,
         "D": 128, "page": 64, "kind": "e4m3", "order": "head", "window": 0},
        # a serving step that mixes prompts' chunks and single tokens, a sliding window, seven queries to a key, padded
        {"name": "attn_b37_n301_l2500_d64", "op": "attn", "B": 37, "n": 301, "L": 2500, "mix": "ragged", "pad": 9, "Hq": 14, "Hkv": 2,
         "D": 64, "page": 16, "kind": "bf16", "order": "token", "window": 1000},
        # a chunk of a prompt over a long context
        {"name": "attn_b1_n512_l32768_d128", "op": "attn", "B": 1, "n": 512, "L": 32768, "mix": "even", "pad": 0, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 32, "kind": "e4m3", "order": "head", "window": 0},
        # a whole prompt: matrix-core bound
        {"name": "attn_b1_n8192_l8192_d128", "op": "attn", "B": 1, "n": 8192, "L": 8192, "mix": "even", "pad": 0, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "kind": "bf16", "order": "head", "window": 0},
        # prompts of wide heads
        {"name": "attn_b4_n1500_l1500_d256", "op": "attn", "B": 4, "n": 1500, "L": 1500, "mix": "ragged", "pad": 0, "Hq": 16, "Hkv": 2,
         "D": 256, "page": 64, "kind": "bf16", "order": "head", "window": 0},
        # what a decoding layer runs for a batch between its products
        {"name": "step_b32_l4000_d128", "op": "step", "B": 32, "n": 1, "L": 4000, "mix": "ragged", "pad": 0, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "kind": "bf16", "order": "head", "window": 0, "rot": 128, "style": "half", "norm": True},
    ]


MOST_WORK = 4 * 128 * 32 * 8192 * 8192 // 2  # multiplications and additions of the largest listed case
MOST_READ = 2 * 2 * 128 * 8 * 500000  # bytes of a listed case's cache
MOST_PLAIN = 2**32  # values that the plain form holds at once


def _log(rng, lo, hi):
    """A whole number, spread evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("rope", "append", "append", "attn", "attn", "attn", "attn", "step"))
    D = rng.choice((64, 128, 128, 128, 256))
    turn = {"rot": rng.choice((D, D, D // 2, D // 4)), "style": rng.choice(("half", "half", "interleaved")), "norm": rng.random() < 0.6}
    if op == "rope":
        H = _log(rng, 1, 64)
        return {"op": op, "T": _log(rng, 1, min(8192, 8192 * 64 * 128 // (H * D))), "H": H, "D": D, **turn, "far": _log(rng, 100, 2000000)}
    Hkv = _log(rng, 1, 16)
    Hq = Hkv * rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 8, 16))
    cache = {"Hq": Hq, "Hkv": Hkv, "D": D, "page": rng.choice((1, 8, 16, 16, 32, 64, 128)), "kind": rng.choice(("bf16", "bf16", "e4m3")),
             "order": rng.choice(("head", "token"))}
    if op == "append":
        return {"op": op, "T": _log(rng, 1, min(8192, 8192 * 80 * 128 // ((Hq + 2 * Hkv) * D))), **cache, **turn, "far": _log(rng, 100, 2000000)}
    how = "decode" if op == "step" else rng.choice(("decode", "decode", "chunk", "prompt"))
    B = _log(rng, 1, 128 if how == "decode" else 24)
    n = 1 if how == "decode" and (op == "step" or rng.random() < 0.7) else _log(rng, 2, 8 if how == "decode" else 8192)
    L = n if how == "prompt" else n + _log(rng, 1, 131072)
    window = rng.choice((0, 0, 0, _log(rng, 16, 4096)))
    while (4 * D * Hq * B * n * L > MOST_WORK or 2 * 2 * D * Hkv * B * L > MOST_READ or B * L * Hkv * D > MOST_PLAIN // 2
           or B * n * L * Hq > MOST_PLAIN // 2):
        if how == "prompt" or n > 512 or L <= n:
            n = max(1, n * 7 // 8)
        L = n if how == "prompt" else max(n, L * 7 // 8)
    case = {"op": op, "B": B, "n": n, "L": L, "mix": rng.choice(("even", "ragged", "ragged")), "pad": rng.choice((0, 0, 0, 5)),
            **cache, "window": window}
    if op == "step":
        case.update(turn, mix="ragged", pad=0)
    return case


def _lengths(case):
    """(new tokens, tokens in all) of each sequence. A ragged batch has one of the full lengths, the others are spread
    over their logarithm; of several, the last is a place of the batch that holds no sequence."""
    B, n, L = case["B"], case["n"], case["L"]
    if case["mix"] == "even":
        return [n] * B, [L] * B
    rng = random.Random(B * 1000003 + n * 8191 + L)
    new = [n] + [_log(rng, 1, n) for _ in range(B - 1)]
    total = [L] + [k if L == n else max(k, _log(rng, max(1, L // 64), L)) for k in new[1:]]
    if B > 2 and case["op"] == "attn":
        new[-1] = total[-1] = 0
    return new, total


def _pages(case):
    """Pages of a cache and of the longest sequence."""
    _, total = _lengths(case)
    P = case["page"]
    return 1 + sum(-(-k // P) for k in total), -(-max(total) // P)


# ---- inputs ------------------------------------------------------------------------------------------------


def _normal(gen, *size):
    return torch.randn(*size, generator=gen, device=DEV)


def _far_channels(gen, x):
    """A few channels that are ten times the others, as keys and queries have them."""
    D = x.shape[-1]
    far = torch.randperm(D, generator=gen, device=DEV)[: max(1, D // 64)]
    x[..., far] *= 10
    return x


def _cache(case, gen, pages, filled):
    """Keys and values [pages, page, Hkv, D], in the memory order of the case; what earlier steps left there if filled."""
    P, Hkv, D = case["page"], case["Hkv"], case["D"]
    both = []
    for scale in (K_SCALE, V_SCALE):
        shape = (pages, P, Hkv, D) if case["order"] == "token" else (pages, Hkv, P, D)
        c = torch.empty(shape, dtype=KINDS[case["kind"]], device=DEV)
        rows = max(1, 2**27 // c[0].numel())
        for i in range(0, pages, rows):  # pieces, so that no copy of the whole in 32 bits is held
            part = c[i : i + rows]
            x = _normal(gen, *part.shape) if filled else torch.zeros(part.shape, device=DEV)
            part.copy_((x / scale if case["kind"] == "e4m3" else x).to(c.dtype))
        both.append(c if case["order"] == "token" else c.transpose(1, 2))
    return both


def _turn_inputs(case, gen, gains):
    rot, D = case["rot"], case["D"]
    s = {"freq": torch.pow(BASE, -torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot).float()}
    for name in gains:
        s[name] = (1 + 0.1 * _normal(gen, D)).to(torch.bfloat16) if case["norm"] else None
    return s


def _append_inputs(case, gen, T):
    """Rows of the layer's first product: queries, keys and values side by side."""
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    row = _normal(gen, T, Hq + 2 * Hkv, D)
    _far_channels(gen, row[:, : Hq + Hkv])
    row = row.to(torch.bfloat16).view(T, (Hq + 2 * Hkv) * D)
    q, k, v = row.split((Hq * D, Hkv * D, Hkv * D), 1)
    s = {"q": q, "k": k, "v": v, "q_out": torch.empty(T, Hq * D, dtype=torch.bfloat16, device=DEV)}
    s.update(_turn_inputs(case, gen, ("gq", "gk")))
    return s


def _attn_inputs(case, gen):
    B, P = case["B"], case["page"]
    new, total = _lengths(case)
    pages, most = _pages(case)
    T = sum(new) + case["pad"]
    start = [sum(new[:b]) for b in range(B + 1)]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    order = torch.randperm(pages - 1, generator=gen, device=DEV).to(torch.int32) + 1  # page 0 belongs to nobody
    need = torch.tensor([-(-k // P) for k in total], device=DEV)
    first = torch.cumsum(need, 0) - need
    at = torch.arange(most, device=DEV)
    table = torch.where(at < need[:, None], order[(first[:, None] + at).clamp(max=max(0, pages - 2))], -1).to(torch.int32)
    s = {"T": T, "pages": pages, "most": most, "start": ints(start), "total": ints(total), "table": table}
    s["kc"], s["vc"] = _cache(case, gen, pages, True)
    s["o"] = torch.zeros(T, case["Hq"] * case["D"], dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros(T, case["Hq"], device=DEV)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, D = case["op"], case["D"]
    s = {"case": case}
    if op == "rope":
        T, H = case["T"], case["H"]
        s["x"] = _far_channels(gen, _normal(gen, T, H, D)).to(torch.bfloat16).view(T, H * D)
        s["y"] = torch.empty_like(s["x"])
        s.update(_turn_inputs(case, gen, ("g",)))
    elif op == "append":
        T, P = case["T"], case["page"]
        s.update(_append_inputs(case, gen, T))
        s["pages"] = 1 + 2 * (-(-T // P))
        s["kc"], s["vc"] = _cache(case, gen, s["pages"], False)
        slots = P + torch.randperm((s["pages"] - 1) * P, generator=gen, device=DEV)[:T]
        slots[torch.rand(T, generator=gen, device=DEV) < 0.03] = -1  # padding of a ragged batch
        s["slots"] = slots
    else:
        s.update(_attn_inputs(case, gen))
        if op == "step":
            s.update(_append_inputs(case, gen, s["T"]))
            s["pos"] = s["total"].long() - 1  # one new token a sequence
            page = s["table"].gather(1, (s["pos"] // case["page"])[:, None])[:, 0]
            s["slots"] = page * case["page"] + s["pos"] % case["page"]
        else:
            s["q"] = (2 * _normal(gen, s["T"], case["Hq"], D)).to(torch.bfloat16).view(s["T"], -1)
    if op in ("rope", "append"):
        s["pos"] = torch.randint(0, case["far"], (case["T"],), generator=gen, device=DEV)
    return s


# ---- one pass ----------------------------------------------------------------------------------------------


def run(s):
    case = s["case"]
    if own:
        return _OWN[case["op"]](s, case)
    return _PLAIN[case["op"]](s, case)


def _plain_turn(x, g, s, case):
    """Heads [T, H, D]: normed, then rotated."""
    x = x.float()
    if g is not None:
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * g.float()
    rot = case["rot"]
    angle = s["pos"].double()[:, None, None] * s["freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    if case["style"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rot:]), 2)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), 3).flatten(2), x[..., rot:]), 2)


def _heads(x, D):
    return x.reshape(x.shape[0], -1, D)


def _plain_rope(s, case):
    y = _plain_turn(_heads(s["x"], case["D"]), s["g"], s, case)
    return y.to(torch.bfloat16).flatten(1)


def _plain_put(cache, slots, x, case):
    """x [T, Hkv, D] at its slots; where a slot is none, what page 0 begins with is written over itself."""
    held = cache.view(torch.uint8) if case["kind"] == "e4m3" else cache
    x = x.clamp(-448, 448).to(cache.dtype).view(torch.uint8) if case["kind"] == "e4m3" else x.to(cache.dtype)
    at = slots.clamp(min=0)
    held[at // case["page"], at % case["page"]] = torch.where((slots >= 0)[:, None, None], x, held[0, 0])


def _plain_append(s, case):
    D = case["D"]
    q = _plain_turn(_heads(s["q"], D), s["gq"], s, case)
    k = _plain_turn(_heads(s["k"], D), s["gk"], s, case)
    v = _heads(s["v"], D).float()
    by_k, by_v = (K_SCALE, V_SCALE) if case["kind"] == "e4m3" else (1.0, 1.0)
    _plain_put(s["kc"], s["slots"], k / by_k, case)
    _plain_put(s["vc"], s["slots"], v / by_v, case)
    return {"q": q.to(torch.bfloat16).flatten(1), "k": s["kc"], "v": s["vc"]}


def _plain_take(cache, s, case, scale):
    """Keys or values of each sequence, padded to the longest: [B, Hkv, L, D]."""
    at = torch.arange(case["L"], device=cache.device)
    page = s["table"].long().clamp(min=0)[:, at // case["page"]]
    held = cache.view(torch.uint8) if case["kind"] == "e4m3" else cache
    x = held[page, at % case["page"]]
    x = x.view(cache.dtype).float() * scale if case["kind"] == "e4m3" else x.float()
    return x.transpose(1, 2)


def _plain_attn(s, case, q=None):
    B, n, L, Hq, Hkv, D = (case[k] for k in ("B", "n", "L", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    q = _heads(s["q"] if q is None else q, D).float()
    k = _plain_take(s["kc"], s, case, K_SCALE)
    v = _plain_take(s["vc"], s, case, V_SCALE)
    start, total = s["start"].long(), s["total"].long()
    count = start[1:] - start[:-1]
    row = torch.arange(n, device=q.device)
    q = q[(start[:-1, None] + row).clamp(max=s["T"] - 1)]  # [B, n, Hq, D]
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    score = (q @ k.transpose(2, 3) * (1 / math.sqrt(D))).view(B, Hkv, G, n, L)
    place = (total - count)[:, None] + row  # [B, n]
    key = torch.arange(L, device=q.device)
    seen = key <= place[:, :, None]
    if case["window"]:
        seen &= key > place[:, :, None] - case["window"]
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    most = score.amax(4, keepdim=True).clamp(min=-1e30)
    e = score.sub_(most).exp_()
    total_e = e.sum(4, keepdim=True)
    o = (e.view(B, Hkv, G * n, L) @ v).view(B, Hkv, G, n, D) / total_e
    lse = most + torch.log(total_e)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq * D)
    lse = lse.permute(0, 3, 1, 2, 4).reshape(B, n, Hq)
    token = torch.arange(s["T"], device=q.device)
    b = torch.searchsorted(start, token, right=True) - 1
    held = (b < B)[:, None]
    b = b.clamp(max=B - 1)
    i = (token - start[b]).clamp(max=n - 1)
    return {"o": torch.where(held, o[b, i], 0.0).to(torch.bfloat16), "lse": torch.where(held, lse[b, i], 0.0)}


def _plain_step(s, case):
    out = _plain_append(s, case)
    return {**out, **_plain_attn(s, case, out["q"])}


def _own_rope(s, case):
    import split_reduction_amd as sk

    sk.skgemm_rope(s["x"], s["g"], s["freq"], s["pos"], s["y"], case["T"], case["H"], case["D"], case["rot"], case["style"], EPS)
    return s["y"]


def _own_append(s, case):
    import split_reduction_amd as sk

    by_k, by_v = (K_SCALE, V_SCALE) if case["kind"] == "e4m3" else (1.0, 1.0)
    sk.skgemm_rope_append(s["q"], s["k"], s["v"], s["gq"], s["gk"], s["freq"], s["pos"], s["slots"], s["q_out"], s["kc"], s["vc"],
                          s["pos"].shape[0], case["Hq"], case["Hkv"], case["D"], s["pages"], case["page"], case["rot"], case["style"],
                          EPS, k_scale=by_k, v_scale=by_v)
    return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}


def _own_attn(s, case, q=None):
    import split_reduction_amd as sk

    by_k, by_v = (K_SCALE, V_SCALE) if case["kind"] == "e4m3" else (1.0, 1.0)
    sk.skgemm_paged_attention(s["q"] if q is None else q, s["kc"], s["vc"], s["table"], s["total"], s["start"], s["o"], s["lse"], s["T"],
                              case["B"], case["n"], case["Hq"], case["Hkv"], case["D"], s["pages"], case["page"], s["most"],
                              1 / math.sqrt(case["D"]), window=case["window"], k_scale=by_k, v_scale=by_v)
    return {"o": s["o"], "lse": s["lse"]}


def _own_step(s, case):
    out = _own_append(s, case)
    return {**out, **_own_attn(s, case, out["q"])}


_PLAIN = {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "step": _plain_step}
_OWN = {"rope": _own_rope, "append": _own_append, "attn": _own_attn, "step": _own_step}


# ---- what a pass cannot do without -------------------------------------------------------------------------


def _size(case):
    return 1 if case["kind"] == "e4m3" else 2


def _append_work(case, T):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    gains = 4 * D if case["norm"] else 0
    return {"bytes": T * (2 * D * (Hq + 2 * Hkv) + 2 * D * Hq + 2 * _size(case) * D * Hkv + 16) + gains + 2 * case["rot"],
            "flops": T * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}


def _attn_work(case):
    Hq, Hkv, D, W = case["Hq"], case["Hkv"], case["D"], case["window"]
    pairs = keys = 0
    new, total = _lengths(case)
    for n, L in zip(new, total):
        pairs += sum(min(p + 1, W or p + 1) for p in range(L - n, L))
        keys += min(L, W + n - 1) if W and n else L if n else 0
    return {"bytes": 2 * _size(case) * D * Hkv * keys + sum(new) * Hq * (4 * D + 4) + 4 * sum(-(-k // case["page"]) for k in total),
            "flops": 4 * D * Hq * pairs}


def work(case):
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        return {"bytes": T * (4 * H * D + 8) + 2 * case["rot"] + (2 * D if case["norm"] else 0),
                "flops": T * H * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    if case["op"] == "append":
        return _append_work(case, case["T"])
    if case["op"] == "attn":
        return _attn_work(case)
    a, b = _append_work(case, sum(_lengths(case)[0])), _attn_work(case)
    return {k: a[k] + b[k] for k in a}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------


def _exact_turn(x, g, s, case):
    """Each pair as a complex number times that of its angle."""
    x = x.double()
    if g is not None:
        x = x / (torch.linalg.vector_norm(x, dim=2, keepdim=True).square() / case["D"] + EPS).sqrt() * g.double()
    rot, half = case["rot"], case["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.outer(s["pos"].double(), s["freq"].double()))[:, None]
    shape = (*x.shape[:2], 2, half) if case["style"] == "half" else (*x.shape[:2], half, 2)
    pairs = x[..., :rot].reshape(shape)
    pairs = pairs.transpose(2, 3) if case["style"] == "half" else pairs
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = y.transpose(2, 3) if case["style"] == "half" else y
    return torch.cat((y.reshape(*x.shape[:2], rot), x[..., rot:]), 2)


def _exact_append(s, case):
    T, D, P = s["pos"].shape[0], case["D"], case["page"]
    by_k, by_v = (K_SCALE, V_SCALE) if case["kind"] == "e4m3" else (1.0, 1.0)
    q, k = (_exact_turn(s[n].reshape(T, -1, D), s["g" + n], s, case) for n in ("q", "k"))
    out = {"q": q.flatten(1)}
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][live].long()
    for name, cache, new in (("k", s["kc"], k / by_k), ("v", s["vc"], s["v"].reshape(T, -1, D).double() / by_v)):
        c = cache.double()
        c.index_put_((at // P, at % P), new[live].clamp(-448, 448) if case["kind"] == "e4m3" else new[live])
        out[name] = c
    return out


def _exact_attn(s, case, caches, q):
    Hq, Hkv, D, P, W = (case[k] for k in ("Hq", "Hkv", "D", "page", "window"))
    o = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], Hq, dtype=torch.float64, device=DEV)
    new, total = _lengths(case)
    first = 0
    for b, (n, L) in enumerate(zip(new, total)):
        ids = s["table"][b, : -(-L // P)].long()
        for h in range(Hq if n else 0):
            k, v = (c[ids, :, h * Hkv // Hq].reshape(-1, D)[:L].double() for c in caches)
            if case["kind"] == "e4m3":
                k, v = k * K_SCALE, v * V_SCALE
            for i in range(0, n, 2048):
                m = min(2048, n - i)
                z = q[first + i : first + i + m, h].double() @ k.T / math.sqrt(D)
                ahead = torch.arange(L, device=DEV)[None] - torch.arange(L - n + i, L - n + i + m, device=DEV)[:, None]
                z[(ahead > 0) | ((ahead <= -W) if W else False)] = -math.inf
                lse[first + i : first + i + m, h] = torch.logsumexp(z, 1)
                o[first + i : first + i + m, h] = torch.softmax(z, 1) @ v
        first += n
    return {"o": o.flatten(1), "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(s["x"].reshape(case["T"], case["H"], case["D"]), s["g"], s, case).flatten(1)
    if case["op"] == "append":
        return _exact_append(s, case)
    if case["op"] == "attn":
        if case["B"] * case["Hq"] > 20000:
            return None
        return _exact_attn(s, case, (s["kc"], s["vc"]), _heads(s["q"], case["D"]))
    out = _exact_append(s, case)
    # the attention reads what was rounded into the cache, and rounded queries
    caches = [out[n].to(s["kc"].dtype) for n in ("k", "v")]
    return {**out, **_exact_attn(s, case, caches, _heads(out["q"].to(torch.bfloat16), case["D"]))}
