"""The operators around the quantised layers and the language-model head, as they are measured.

Four operators: the root-mean-square norm with the residual's addition and an 8-bit (or bf16) output, the
product of 8-bit integers with a scale for each token and each output channel, the log probabilities of given
tokens with entropy and the best alternatives, and the gradient of those log probabilities and entropies to the
logits. ``run`` makes one pass through one of them (``layer``: the norm and the product that reads it).

With ``own`` false the pass is the plain form, elementary torch operations in 32 bits, rounded once at the end;
with ``own`` true it is the call a program makes of ``split_reduction_amd``.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ---------------------------------------------------------------------------------------------


def listed():
    return [
        # one decode step of one sequence: launch latency
        {"name": "norm_t1_h7168", "op": "norm", "T": 1, "H": 7168, "residual": True, "out": "e4m3"},
        # a long prompt's rows: memory traffic
        {"name": "norm_t8192_h7168", "op": "norm", "T": 8192, "H": 7168, "residual": True, "out": "e4m3"},
        # norm, 8-bit codes and the wide projection that reads them, a full decode batch
        {"name": "layer_t128_h16384", "op": "layer", "T": 128, "H": 16384, "N": 16384, "residual": True, "out": "bf16"},
        # one token through a projection of a layer: latency, few rows
        {"name": "i8_t1_k7168_n2048", "op": "i8", "T": 1, "K": 7168, "N": 2048, "out": "bf16"},
        # a decode batch through a wide projection: the weights' traffic
        {"name": "i8_t32_k7168_n18432", "op": "i8", "T": 32, "K": 7168, "N": 18432, "out": "bf16"},
        # a ragged prompt and an output width that is no multiple of a tile
        {"name": "i8_t509_k7168_n4100", "op": "i8", "T": 509, "K": 7168, "N": 4100, "out": "f32"},
        # prompt processing: matrix-core bound
        {"name": "i8_t4096_k7168_n18432", "op": "i8", "T": 4096, "K": 7168, "N": 18432, "out": "bf16"},
        # one sampled token with its alternatives, as a serving interface reports them: latency
        {"name": "logp_t1_v131072", "op": "logp", "T": 1, "V": 131072, "k": 20, "type": "bf16", "banned": 0.0, "scale": 1.0},
        # a decode batch under a grammar that bans most tokens, an odd vocabulary
        {"name": "logp_t67_v50001", "op": "logp", "T": 67, "V": 50001, "k": 5, "type": "f32", "banned": 0.9, "scale": 1.25},
        # scoring a long prompt: memory traffic
        {"name": "logp_t4096_v131072", "op": "logp", "T": 4096, "V": 131072, "k": 8, "type": "bf16", "banned": 0.0, "scale": 1.0},
        # a small update batch in 32 bits
        {"name": "grad_t64_v32001", "op": "grad", "T": 64, "V": 32001, "type": "f32", "banned": 0.0, "scale": 1.0},
        # an update batch of a policy trained on its own log probabilities
        {"name": "grad_t4096_v131072", "op": "grad", "T": 4096, "V": 131072, "type": "bf16", "banned": 0.0, "scale": 0.8},
    ]


def _log(rng, lo, hi):
    """A whole number, spread evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("norm", "layer", "i8", "i8", "logp", "logp", "grad"))
    if op == "norm":
        H = 8 * _log(rng, 64, 2048)
        return {"op": op, "T": _log(rng, 1, min(8192, 8192 * 7168 // H)), "H": H, "residual": rng.random() < 0.7,
                "out": rng.choice(("e4m3", "e4m3", "bf16"))}
    if op in ("layer", "i8"):
        K = 16 * _log(rng, 16, 1024)
        N = _log(rng, 64, 18432)
        T = _log(rng, 1, min(4096, 4096 * 7168 * 18432 // (K * N)))
        out = rng.choice(("bf16", "bf16", "f32"))
        if op == "layer":
            return {"op": op, "T": T, "H": K, "N": N, "residual": rng.random() < 0.7, "out": "bf16"}
        return {"op": op, "T": T, "K": K, "N": N, "out": out}
    V = _log(rng, 1000, 262144)
    T = _log(rng, 1, min(4096, 4096 * 131072 // (2 * V)))
    case = {"op": op, "T": T, "V": V, "type": rng.choice(("bf16", "f32")), "banned": rng.choice((0.0, 0.0, 0.5, 0.95)),
            "scale": rng.choice((1.0, 1.0, 0.7, 1.6))}
    if op == "logp":
        case["k"] = _log(rng, 1, 64)
    return case


# ---- inputs ------------------------------------------------------------------------------------------------


def _codes(gen, rows, cols):
    """8-bit codes of normal values, the largest of a row near 127."""
    z = torch.randn(rows, cols, generator=gen, device=DEV)
    return z.mul_(127 / 4.5).round_().clamp_(-127, 127).to(torch.int8)


def _norm_inputs(case, gen):
    T, H = case["T"], case["H"]
    x = torch.randn(T, H, generator=gen, device=DEV)
    r = torch.randn(T, H, generator=gen, device=DEV) * 2
    far = torch.randperm(H, generator=gen, device=DEV)[: max(1, H // 100)]
    r[:, far] *= 10  # the few channels that a residual stream holds at ten times the others
    s = {"x": x.to(torch.bfloat16), "r": r.to(torch.bfloat16) if case["residual"] else None,
         "g": (1 + 0.1 * torch.randn(H, generator=gen, device=DEV)).to(torch.bfloat16)}
    s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    T, op = case["T"], case["op"]
    s = {"case": case}
    if op in ("norm", "layer"):
        s.update(_norm_inputs(case, gen))
        H = case["H"]
        kind = {"e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16}[case["out"]] if op == "norm" else torch.int8
        s["y"] = torch.empty(T, H, dtype=kind, device=DEV)
        s["ys"] = torch.empty(T, dtype=torch.float32, device=DEV)
    if op in ("layer", "i8"):
        K, N = case["H"] if op == "layer" else case["K"], case["N"]
        s["w"] = _codes(gen, N, K)
        s["ws"] = (0.02 * 4.5 / 127) * (0.5 + torch.rand(N, generator=gen, device=DEV))
        s["c"] = torch.empty(T, N, dtype=TYPES[case["out"]], device=DEV)
        if op == "i8":
            s["x"] = _codes(gen, T, K)
            s["xs"] = (4.5 / 127) * (0.5 + torch.rand(T, generator=gen, device=DEV))
    if op in ("logp", "grad"):
        V, kind = case["V"], TYPES[case["type"]]
        z = torch.randn(T, V, generator=gen, device=DEV).mul_(2.5)
        likely = torch.randint(0, V, (T, 8), generator=gen, device=DEV)
        z.scatter_add_(1, likely, 4 + 10 * torch.rand(T, 8, generator=gen, device=DEV))
        if case["banned"]:
            z.masked_fill_(torch.rand(T, V, generator=gen, device=DEV) < case["banned"], -math.inf)
        z[:, :1] = torch.randn(T, 1, generator=gen, device=DEV)  # one token at least stays allowed
        s["z"] = z.to(kind)
        del z
        pick = torch.randint(0, 8, (T, 1), generator=gen, device=DEV)
        tokens = likely.gather(1, pick)[:, 0]
        tokens[torch.rand(T, generator=gen, device=DEV) < 0.05] = -1  # padding of a ragged batch
        s["tokens"] = tokens
        f32 = lambda *n: torch.empty(*n, dtype=torch.float32, device=DEV)  # noqa: E731
        if op == "logp":
            s.update(logp=f32(T), entropy=f32(T), lse=f32(T), top=f32(T, case["k"]),
                     ids=torch.empty(T, case["k"], dtype=torch.int64, device=DEV))
        else:
            a = s["z"].float() * case["scale"]
            s["lse"] = torch.logsumexp(a, 1)
            p = torch.exp(a - s["lse"][:, None])
            s["entropy"] = s["lse"] - (p * a.clamp(min=-1e30)).sum(1)
            s["g_logp"] = torch.randn(T, generator=gen, device=DEV)
            s["g_entropy"] = 0.05 * torch.randn(T, generator=gen, device=DEV)
            s["dz"] = torch.empty_like(s["z"])
    return s


# ---- one pass ----------------------------------------------------------------------------------------------


def run(s):
    case = s["case"]
    if own:
        return _OWN[case["op"]](s, case)
    return _PLAIN[case["op"]](s, case)


def _plain_normed(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["g"].float()
    return h, y


def _plain_norm(s, case):
    h, y = _plain_normed(s)
    out = {"sum": h.to(torch.bfloat16)} if s["r"] is not None else {}
    if case["out"] == "bf16":
        return {**out, "y": y.to(torch.bfloat16)}
    scale = y.abs().amax(1, keepdim=True) / 448
    return {**out, "y": (y / scale).clamp(-448, 448).to(torch.float8_e4m3fn), "scale": scale[:, 0]}


def _plain_product(x, xs, w, ws, kind):
    return ((x @ w.float().t()) * xs[:, None] * ws).to(kind)


def _plain_layer(s, case):
    h, y = _plain_normed(s)
    out = {"sum": h.to(torch.bfloat16)} if s["r"] is not None else {}
    scale = y.abs().amax(1) / 127
    codes = torch.round(y / scale[:, None])
    return {**out, "c": _plain_product(codes, scale, s["w"], s["ws"], torch.bfloat16)}


def _plain_i8(s, case):
    return _plain_product(s["x"].float(), s["xs"], s["w"], s["ws"], TYPES[case["out"]])


def _plain_logp(s, case):
    z = s["z"].float()
    d = z * case["scale"]
    most = d.amax(1, keepdim=True)
    d = d - most
    e = torch.exp(d)
    total = e.sum(1)
    log_total = torch.log(total)
    entropy = log_total - torch.where(e > 0, e * d, 0.0).sum(1) / total
    tokens = s["tokens"]
    given = d.gather(1, tokens.clamp(min=0)[:, None])[:, 0] - log_total
    # the best k, of equal ones the lowest index: order by (value, -index) in one whole number
    bits = z.view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)  # as the values are ordered, -0 with 0
    columns = torch.arange(z.shape[1], device=z.device)
    ids = torch.topk(order * 2**20 + (2**20 - 1 - columns), case["k"], dim=1).values
    ids = 2**20 - 1 - (ids & (2**20 - 1))
    return {"logp": torch.where(tokens >= 0, given, 0.0), "entropy": entropy, "lse": most[:, 0] + log_total,
            "top": d.gather(1, ids) - log_total[:, None], "ids": ids}


def _plain_grad(s, case):
    a = s["z"].float() * case["scale"]
    lp = a - s["lse"][:, None]
    p = torch.exp(lp)
    tokens = s["tokens"]
    g = torch.where(tokens >= 0, s["g_logp"], 0.0)
    d = -g[:, None] * p - s["g_entropy"][:, None] * torch.where(p > 0, p * (lp + s["entropy"][:, None]), 0.0)
    d.scatter_add_(1, tokens.clamp(min=0)[:, None], g[:, None])
    return (d * case["scale"]).to(s["z"].dtype)


def _own_norm(s, case):
    import split_reduction_amd as sk

    out = {"sum": s["sum"]} if s["r"] is not None else {}
    if case["out"] == "bf16":
        sk.skgemm_rmsnorm(s["x"], s["r"], s["g"], s["sum"], s["y"], None, case["T"], case["H"], EPS, "bf16")
        return {**out, "y": s["y"]}
    sk.skgemm_rmsnorm(s["x"], s["r"], s["g"], s["sum"], s["y"], s["ys"], case["T"], case["H"], EPS, "e4m3")
    return {**out, "y": s["y"], "scale": s["ys"]}


def _own_layer(s, case):
    import split_reduction_amd as sk

    sk.skgemm_rmsnorm(s["x"], s["r"], s["g"], s["sum"], s["y"], s["ys"], case["T"], case["H"], EPS, "i8")
    sk.skgemm_i8(s["w"], s["ws"], s["y"], s["ys"], s["c"], case["T"], case["N"], case["H"])
    return {**({"sum": s["sum"]} if s["r"] is not None else {}), "c": s["c"]}


def _own_i8(s, case):
    import split_reduction_amd as sk

    sk.skgemm_i8(s["w"], s["ws"], s["x"], s["xs"], s["c"], case["T"], case["N"], case["K"])
    return s["c"]


def _own_logp(s, case):
    import split_reduction_amd as sk

    sk.skgemm_logprobs(s["z"], s["tokens"], s["logp"], s["entropy"], s["lse"], s["top"], s["ids"], case["T"], case["V"],
                       case["k"], case["scale"])
    return {"logp": s["logp"], "entropy": s["entropy"], "lse": s["lse"], "top": s["top"], "ids": s["ids"]}


def _own_grad(s, case):
    import split_reduction_amd as sk

    sk.skgemm_logprobs_grad(s["z"], s["tokens"], s["lse"], s["entropy"], s["g_logp"], s["g_entropy"], s["dz"], case["T"],
                            case["V"], case["scale"])
    return s["dz"]


_PLAIN = {"norm": _plain_norm, "layer": _plain_layer, "i8": _plain_i8, "logp": _plain_logp, "grad": _plain_grad}
_OWN = {"norm": _own_norm, "layer": _own_layer, "i8": _own_i8, "logp": _own_logp, "grad": _own_grad}


# ---- what a pass cannot do without -------------------------------------------------------------------------


def work(case):
    T, op = case["T"], case["op"]
    if op in ("norm", "layer"):
        H = case["H"]
        rows = 2 * T * H + (4 * T * H if case["residual"] else 0) + 2 * H
        if op == "norm":
            size = 1 if case["out"] == "e4m3" else 2
            return {"bytes": rows + size * T * H + (4 * T if size == 1 else 0), "flops": 6 * T * H}
        N = case["N"]
        return {"bytes": rows + N * H + 4 * N + 2 * T * N, "flops": 2 * T * N * H + 6 * T * H}
    if op == "i8":
        K, N = case["K"], case["N"]
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": N * K + T * K + 4 * (N + T) + size * T * N, "flops": 2 * T * N * K}
    V, size = case["V"], 4 if case["type"] == "f32" else 2
    if op == "logp":
        return {"bytes": size * T * V + 20 * T + 12 * T * case["k"], "flops": 6 * T * V}
    return {"bytes": 2 * size * T * V + 24 * T, "flops": 8 * T * V}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "layer"):
        h = s["x"].double()
        if case["residual"]:
            h += s["r"].double()
        length = torch.linalg.vector_norm(h, dim=1, keepdim=True)
        y = s["g"].double() * (h / torch.sqrt(length**2 / case["H"] + EPS))
        out = {"sum": h} if case["residual"] else {}
        if op == "norm" and case["out"] == "bf16":
            return {**out, "y": y}
        top = 127.0 if op == "layer" else 448.0
        step = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / top
        codes = y / step[:, None]
        if op == "norm":
            return {**out, "y": codes, "scale": step}
        s["x"], s["xs"] = torch.floor(codes + 0.5), step
        return {**out, "c": _exact_product(s)}
    if op == "i8":
        return _exact_product(s)
    return _exact_logp(s, case) if op == "logp" else _exact_grad(s, case)


def _exact_product(s):
    x, w = s["x"].double() * s["xs"].double()[:, None], s["w"].double() * s["ws"].double()[:, None]
    return torch.matmul(x, w.t())


def _by_rows(s, case, f):
    """`f` of 256 rows at a time, joined: 64-bit copies of the whole logits need not be held."""
    parts = [f(slice(i, i + 256)) for i in range(0, case["T"], 256)]
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


def _exact_logp(s, case):
    def rows(at):
        a = s["z"][at].double() * case["scale"]
        lse = torch.logsumexp(a, 1)
        lp = a - lse[:, None]
        entropy = torch.special.entr(lp.exp()).sum(1)
        tokens = s["tokens"][at]
        given = lp.gather(1, tokens.clamp(min=0)[:, None])[:, 0].masked_fill(tokens < 0, 0.0)
        ids = torch.sort(s["z"][at].double(), dim=1, descending=True, stable=True).indices[:, : case["k"]]
        return {"logp": given, "entropy": entropy, "lse": lse, "top": lp.gather(1, ids), "ids": ids}

    return _by_rows(s, case, rows)


def _exact_grad(s, case):
    def rows(at):
        # with the lse and entropy that the call is given; both are rounded to 32 bits
        lp = s["z"][at].double() * case["scale"] - s["lse"][at].double()[:, None]
        p = lp.exp()
        tokens = s["tokens"][at]
        hit = torch.arange(case["V"], device=DEV) == tokens[:, None]
        g = s["g_logp"][at].double().masked_fill(tokens < 0, 0.0)
        d = g[:, None] * (hit.double() - p)
        d += s["g_entropy"][at].double()[:, None] * (torch.special.entr(p) - p * s["entropy"][at].double()[:, None])
        return {"d": d * case["scale"]}

    return _by_rows(s, case, rows)["d"]
