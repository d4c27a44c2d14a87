"""More operators of an expert layer, as they are measured: what each call gets,
what it returns and what it cannot do without.

Five operators, each reached through the package's own entry points:

* scores    the router's selection by scores: sigmoid or softmax scores of E
            logits, chosen by score plus a balancing bias within the best
            groups of experts, weighted by the scores alone, and the order
            that groups the token-expert pairs by expert; for training also
            the gradient of the logits;
* quantize  rows to microscaled 4-bit floating point (blocks of 32 values with
            a power-of-two scale, elements of two exponent bits and one
            mantissa bit) and back to the values the codes stand for;
* product   the matrix product of two such operands: grouped by expert with
            ragged sizes, and dense from BF16 rows, which are quantised in the
            call;
* ffn       a serving step's gated feed-forward block of E experts on such
            weights, from BF16 rows and router logits to BF16 rows;
* gate      the gated activation of a training step's experts with its row
            weights, which keeps its inputs in 8 bits, and its backward pass
            from what was kept.

With `own` false, run() computes the same from elementary torch operations in
FP32 (the selection's comparisons in 64 bits), rounded once at the end.  Sizes
are those of the package's workloads (E = 8 and 32 experts, d_model 2048,
gate_up 1536, down 768, 16384 tokens on 256 experts, 131072 rows, the
4096 x 4096 projection), single tokens and batches of a few, and odd sizes
between them.
"""
import math

import torch

own = False

# the largest product of the listed cases: rows x output channels x reduction
MOST_WORK = 131072 * 2048 * 1536

# magnitudes of the 4-bit codes 0 .. 7 (code 8 and above: the same, negative)
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

BLOCK8 = 128   # columns that share a scale in the kept 8-bit activations


def listed():
    return [
        # one token of a decoding step: sigmoid scores with a bias, 4 of 8 groups
        {"name": "scores_token", "op": "scores", "T": 1, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "best": 2, "renormalize": True, "scale": 2.5, "grad": False, "padded": 0.0},
        # a prompt of odd length on 100 experts in 4 groups by their best softmax score, an eighth of it padding
        {"name": "scores_prompt", "op": "scores", "T": 2039, "E": 100, "k": 6, "score": "softmax", "bias": False, "groups": 4,
         "top_groups": 2, "best": 1, "renormalize": False, "scale": 1.0, "grad": True, "padded": 0.125},
        # a training step's 16384 tokens on 256 experts, forward and the logits' gradient
        {"name": "scores_train", "op": "scores", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "best": 2, "renormalize": True, "scale": 2.5, "grad": True, "padded": 0.0},
        # the activations of a decoding step for 16 sequences, there and back
        {"name": "quantize_decode", "op": "quantize", "T": 16, "K": 2048, "dtype": "bf16"},
        # the gate_up weights of 32 experts as they are loaded, there and back
        {"name": "quantize_weights", "op": "quantize", "T": 49152, "K": 2048, "dtype": "fp32"},
        # one decoded token through the square projection, from BF16
        {"name": "product_token", "op": "product", "E": 0, "M": 1, "N": 4096, "K": 4096, "skew": 0.0, "empty": 0, "out": "bf16"},
        # a Zipf-routed prompt on the down shape, two experts without rows, FP32 output
        {"name": "product_ragged", "op": "product", "E": 32, "M": 16411, "N": 2048, "K": 768, "skew": 1.2, "empty": 2, "out": "fp32"},
        # the gate_up product at its full size
        {"name": "product_full", "op": "product", "E": 8, "M": 131072, "N": 1536, "K": 2048, "skew": 0.0, "empty": 0, "out": "bf16"},
        # a decoding step of 8 sequences through the whole block
        {"name": "ffn_decode", "op": "ffn", "T": 8, "E": 32, "k": 4, "H": 2048, "I": 768},
        # 16384 prompt tokens through the whole block, 8 experts each
        {"name": "ffn_prompt", "op": "ffn", "T": 16384, "E": 32, "k": 8, "H": 2048, "I": 768},
        # a short odd batch through the activation and its backward pass
        {"name": "gate_odd", "op": "gate", "T": 517, "k": 3, "I": 776},
        # a training step's 131072 rows, forward and backward
        {"name": "gate_train", "op": "gate", "T": 16384, "k": 8, "I": 768},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scores", "quantize", "product", "ffn", "gate"])
    if op == "scores":
        groups, size = rng.choice([(1, 8), (1, 57), (4, 16), (4, 25), (8, 8), (8, 32), (5, 12), (16, 16)])
        top = rng.randint(1, groups)
        return {"op": op, "T": _log(rng, 1, 16384) | 1, "E": groups * size, "k": rng.randint(1, min(8, top * size)),
                "score": rng.choice(["sigmoid", "sigmoid", "softmax"]), "bias": rng.random() < 0.6, "groups": groups,
                "top_groups": top, "best": rng.choice([1, 2]), "renormalize": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "grad": rng.random() < 0.5, "padded": rng.choice([0.0, 0.2])}
    if op == "quantize":
        K = 32 * rng.randint(4, 128)
        return {"op": op, "T": _log(rng, 1, min(49152, 49152 * 2048 // K)) | 1, "K": K, "dtype": rng.choice(["bf16", "fp32"])}
    if op == "product":
        E = rng.choice([0, 1, 8, 32, 57])
        N, K = 8 * (2 * rng.randint(32, 200) + 1), 32 * (2 * rng.randint(4, 50) + 1)
        most = min(65536, MOST_WORK // (N * K))
        return {"op": op, "E": E, "M": _log(rng, 1, most) | 1, "N": N, "K": K, "skew": rng.choice([0.0, 1.2]),
                "empty": 2 if E > 8 else 0, "out": rng.choice(["bf16", "fp32"])}
    if op == "ffn":
        return {"op": op, "T": _log(rng, 1, 8000) | 1, "E": rng.choice([8, 32, 57]), "k": rng.randint(1, 8),
                "H": 32 * (2 * rng.randint(8, 31) + 1), "I": 32 * (2 * rng.randint(4, 11) + 1)}
    return {"op": op, "T": _log(rng, 1, 16000) | 1, "k": rng.randint(1, 8), "I": 8 * (2 * rng.randint(16, 47) + 1)}


# ---- inputs -------------------------------------------------------------------

def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _logits(g, case):
    """Router logits: normal, with a bias per expert (some are busier)."""
    logits = _normal(g, case["T"], case["E"]) + 0.5 * _normal(g, 1, case["E"])
    padded = case.get("padded", 0.0)
    if padded:   # padding tokens: every expert masked
        logits.masked_fill_(torch.rand((case["T"], 1), generator=g, device="cuda") < padded, -math.inf)
    return logits


def _counts(g, E, M, skew, empty):
    """Rows of each expert: shares rank^-skew over the experts that have any."""
    share = torch.arange(1, E - empty + 1, dtype=torch.float64) ** -skew
    at = torch.multinomial(share, M, replacement=True, generator=g)
    return torch.bincount(torch.randperm(E, generator=g)[at], minlength=E)


def _packed(g, *shape):
    """Codes and scales of normal rows in the package's layout: two codes a
    byte, the even column in the low half; the scales of 256 columns (8 blocks
    of 32) side by side, row after row, [ceil(K / 256), rows.., 8]."""
    rows, K = shape[:-1], shape[-1]
    codes, scale = _plain_codes(torch.randn(shape, generator=g, device="cuda").reshape(-1, K))
    codes = (codes[:, 0::2] | codes[:, 1::2] << 4).reshape(*rows, K // 2)
    blocks = -(-K // 256)
    scale = torch.nn.functional.pad(scale, (0, 8 * blocks - K // 32)).reshape(-1, blocks, 8)
    return codes, scale.permute(1, 0, 2).contiguous().reshape(blocks, *rows, 8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)
    s = dict(case)
    if case["op"] == "scores":
        s["logits"] = _logits(g, case)
        # balancing biases move by a fixed step at a time
        s["b"] = torch.round(_normal(g, case["E"], std=30.0)) * 0.001 if case["bias"] else None
        if case["grad"]:
            s["dweights"] = _normal(g, case["T"], case["k"])
    elif case["op"] == "quantize":
        s["x"] = _normal(g, case["T"], case["K"], dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    elif case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        if case["E"] == 0:
            s["x"] = _normal(g, M, K, dtype=torch.bfloat16)
            s["w"], s["ws"] = _packed(g, N, K)
        else:
            s["x"], s["xs"] = _packed(g, M, K)
            s["w"], s["ws"] = _packed(g, case["E"], N, K)
            counts = _counts(h, case["E"], M, case["skew"], case["empty"])
            s["counts"] = counts.tolist()
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32).cuda()
    elif case["op"] == "ffn":
        s["logits"] = _logits(g, case)
        s["b"] = torch.round(_normal(g, case["E"], std=30.0)) * 0.001
        s["x"] = _normal(g, case["T"], case["H"], dtype=torch.bfloat16)
        s["w1"], s["s1"] = _packed(g, case["E"], 2 * case["I"], case["H"])
        s["w2"], s["s2"] = _packed(g, case["E"], case["H"], case["I"])
    else:
        T, k, I = case["T"], case["k"], case["I"]
        # k distinct experts of 64 for each token, grouped by expert
        experts = torch.rand((T, 64), generator=g, device="cuda").argsort(1)[:, :k]
        s["positions"] = experts.flatten().argsort(stable=True).argsort().to(torch.int32).reshape(T, k)
        s["weights"] = torch.softmax(_normal(g, T, k), 1)
        s["gu"] = _normal(g, T * k, 2 * I, dtype=torch.bfloat16)
        s["dh"] = _normal(g, T * k, I, dtype=torch.bfloat16)
    return s


# ---- the plain form -------------------------------------------------------------

def _plain_scores(logits, bias, s):
    """(experts, weights, offsets, positions); comparisons on 64-bit scores."""
    T, E = logits.shape
    l = logits.double()
    masked = l == -math.inf
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        most = l.amax(1, keepdim=True)
        p = torch.exp(torch.where(masked, -math.inf, l - torch.where(most == -math.inf, 0.0, most)))
        total = p.sum(1, keepdim=True)
        score = p / torch.where(total == 0, 1.0, total)
    value = score if bias is None else score + bias.double()
    value = torch.where(masked, -math.inf, value)
    if bias is None and s["groups"] == 1:
        value = l
    elif s["groups"] > 1:
        by_group = value.reshape(T, s["groups"], -1)
        best = torch.sort(by_group, dim=2, descending=True)[0][:, :, :s["best"]]
        rank = torch.where(best == -math.inf, 0.0, best).sum(2)
        rank = torch.where(best[:, :, 0] == -math.inf, -math.inf, rank)
        kept = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :s["top_groups"]]
        keep = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, kept, True)
        # an expert of a group that is not kept comes after the masked ones of those that are
        order = keep[:, :, None].expand_as(by_group).reshape(T, E)
        first = torch.sort(value, dim=1, descending=True, stable=True)[1]
        second = torch.sort(order.gather(1, first).to(torch.int8), dim=1, descending=True, stable=True)[1]
        experts = first.gather(1, second)[:, :s["k"]]
    if s["groups"] == 1:
        experts = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :s["k"]]
    weights = torch.where(masked, 0.0, score).gather(1, experts)
    if s["renormalize"]:
        total = weights.sum(1, keepdim=True)
        weights = weights / torch.where(total == 0, 1.0, total)
    weights = (weights * s["scale"]).float()
    order = torch.sort(experts.reshape(-1), stable=True)[1]
    positions = torch.empty_like(order)
    positions[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=logits.device)
    offsets[1:] = torch.bincount(experts.reshape(-1), minlength=E).cumsum(0)
    return experts.to(torch.int32), weights, offsets.to(torch.int32), positions.reshape(experts.shape).to(torch.int32)


def _plain_scores_grad(dweights, logits, experts, weights, s):
    at, c = experts.long(), s["scale"]
    inner = (weights * dweights).sum(1, keepdim=True)
    if s["score"] == "softmax" and not s["renormalize"]:
        most = logits.amax(1, keepdim=True)
        p = torch.exp(torch.where(most == -math.inf, -math.inf, logits - most))
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total == 0, 1.0, total)
        return p * (torch.zeros_like(logits).scatter_(1, at, c * dweights) - inner)
    d = weights * (dweights - inner / c) if s["renormalize"] else weights * dweights
    if s["score"] == "sigmoid":
        d = d / (1 + torch.exp(logits.gather(1, at)))
    return torch.zeros_like(logits).scatter_(1, at, torch.where(weights == 0, 0.0, d))


def _plain_codes(x):
    """(codes [T, K] in 0 .. 15, scale bytes [T, K / 32])."""
    T, K = x.shape
    x = x.float().reshape(T, K // 32, 32)
    most = x.abs().amax(2)
    byte = (torch.frexp(most)[1] - 3 + 127).clamp(0, 254) * (most > 0)
    a = torch.ldexp(x, (127 - byte)[:, :, None])
    mag = a.abs()
    code = torch.where(mag < 2, torch.round(2 * mag), torch.where(mag < 4, torch.round(mag) + 2, torch.round(mag / 2) + 4))
    code = code.clamp(max=7).to(torch.uint8) + 8 * (a < 0).to(torch.uint8)
    return code.reshape(T, K), byte.to(torch.uint8)


def _plain_values(codes, scale):
    """FP32 values of codes [T, K] (one a byte) and scale bytes [T, K / 32]."""
    T, K = codes.shape
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=codes.device)
    return torch.ldexp(table[codes.long()].reshape(T, K // 32, 32), (scale.int() - 127)[:, :, None]).reshape(T, K)


def _plain_unpack(codes, scale):
    """FP32 values [.., K] of the package's layout."""
    rows, K = codes.shape[:-1], 2 * codes.shape[-1]
    each = torch.stack([codes & 15, codes >> 4], -1).reshape(-1, K)
    scale = scale.reshape(scale.shape[0], -1, 8).permute(1, 0, 2).reshape(-1, 8 * scale.shape[0])[:, :K // 32]
    return _plain_values(each, scale).reshape(*rows, K)


def _plain_rounded(x):
    return _plain_values(*_plain_codes(x))


def _plain_grouped(x, w, counts):
    return torch.cat([a @ b.T for a, b in zip(x.split(counts), w)])


def _ffn_scores(s):
    return dict(score="sigmoid", groups=1, top_groups=1, best=1, renormalize=True, scale=2.5, k=s["k"])


def _plain_ffn(s):
    experts, weights, offsets, positions = _plain_scores(s["logits"], s["b"], _ffn_scores(s))
    counts = (offsets[1:] - offsets[:-1]).tolist()
    at = positions.long()
    token = torch.empty(at.numel(), dtype=torch.int64, device=at.device)
    token[at.reshape(-1)] = torch.arange(at.shape[0], device=at.device).repeat_interleave(at.shape[1])
    y = _plain_grouped(_plain_rounded(s["x"])[token], _plain_unpack(s["w1"], s["s1"]), counts)
    gate, up = y[:, :s["I"]], y[:, s["I"]:]
    y = _plain_grouped(_plain_rounded(gate / (1 + torch.exp(-gate)) * up), _plain_unpack(s["w2"], s["s2"]), counts)
    return (y[at] * weights[:, :, None]).sum(1).to(torch.bfloat16)


def _plain_kept(x):
    """The values that 8-bit codes of blocks of BLOCK8 columns stand for."""
    n = x.shape[1]
    x = torch.nn.functional.pad(x, (0, -n % BLOCK8)).reshape(x.shape[0], -1, BLOCK8)
    most = x.abs().amax(2, keepdim=True)
    codes = torch.round(x * 127 / torch.where(most == 0, 1.0, most))
    return (codes * (most / 127)).reshape(x.shape[0], -1)[:, :n]


def _plain_gate(s):
    I, at = s["I"], s["positions"].long()
    w = torch.empty((at.numel(), 1), device=at.device)
    w[at.reshape(-1)] = s["weights"].reshape(-1, 1)
    g, u = s["gu"].float().split(I, 1)
    out = [(w * (g / (1 + torch.exp(-g)) * u)).to(torch.bfloat16)]
    g, u, dh = _plain_kept(g), _plain_kept(u), s["dh"].float()
    sig = 1 / (1 + torch.exp(-g))
    h = g * sig * u
    d = w * dh
    dgu = torch.cat([d * u * sig * (1 + g * (1 - sig)), d * g * sig], 1)
    return out + [dgu.to(torch.bfloat16), (w * h).to(torch.bfloat16), (dh * h).sum(1)[at]]


def _plain(s):
    if s["op"] == "scores":
        got = _plain_scores(s["logits"], s["b"], s)
        if s["grad"]:
            got += (_plain_scores_grad(s["dweights"], s["logits"], got[0], got[1], s),)
        return got
    if s["op"] == "quantize":
        return _plain_rounded(s["x"]).to(torch.bfloat16)
    if s["op"] == "product":
        dt = torch.bfloat16 if s["out"] == "bf16" else torch.float32
        w = _plain_unpack(s["w"], s["ws"])
        if s["E"] == 0:
            return (_plain_rounded(s["x"]) @ w.T).to(dt)
        return _plain_grouped(_plain_unpack(s["x"], s["xs"]), w, s["counts"]).to(dt)
    return _plain_ffn(s) if s["op"] == "ffn" else _plain_gate(s)


# ---- the framework's operators -------------------------------------------------

def _own(s):
    import dense_ragged_grouped_amd as drgg
    from dense_ragged_grouped_amd import moe
    if s["op"] == "scores":
        scoring = drgg.Scoring(s["score"], bias=s["b"], groups=s["groups"], top_groups=s["top_groups"], best=s["best"],
                               renormalize=s["renormalize"], scale=s["scale"])
        r = drgg.moe_route_scores(s["logits"], s["k"], scoring)
        got = (r.experts, r.weights, r.group_offsets, r.positions)
        if s["grad"]:
            got += (drgg.moe_route_scores_grad(s["dweights"], s["logits"], r.experts, r.weights, scoring),)
        return got
    if s["op"] == "quantize":
        return drgg.dequantize_mxfp4(*drgg.quantize_mxfp4(s["x"]))
    if s["op"] == "product":
        dt = torch.bfloat16 if s["out"] == "bf16" else torch.float32
        if s["E"] == 0:
            x, xs = drgg.quantize_mxfp4(s["x"])
            return drgg.gemm_mxfp4(x, xs, s["w"], s["ws"], out_dtype=dt)
        return drgg.grouped_gemm_mxfp4(s["x"], s["xs"], s["w"], s["ws"], s["offsets"], out_dtype=dt)
    if s["op"] == "ffn":
        scoring = drgg.Scoring("sigmoid", bias=s["b"], scale=2.5)
        return moe.ffn_mxfp4(s["x"], s["logits"], s["w1"], s["s1"], s["w2"], s["s2"], s["k"], scoring=scoring)
    h, kept, scale = drgg.moe_gate_int8(s["gu"], s["positions"], s["weights"])
    return [h, *drgg.moe_gate_int8_grad(s["dh"], kept, scale, s["positions"], s["weights"])]


def run(state):
    return _own(state) if own else _plain(state)


# ---- the same from the definitions, in 64 bits ------------------------------------

def _exact_choice(l, b, s):
    """The k experts of each token by taking the best one k times."""
    T, E = l.shape
    best_of = l.max(1, keepdim=True).values
    none = torch.isinf(best_of) & (best_of < 0)
    score = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.where(none, 0.0, torch.exp(l - torch.logsumexp(l, 1, True)))
    value = l.clone()
    if b is not None or s["groups"] > 1:
        value = score + (0 if b is None else b.double())
        value[l == -math.inf] = -math.inf
    index = torch.arange(E, device=l.device)
    open_ = torch.ones((T, E), dtype=torch.bool, device=l.device)
    rows = torch.arange(T, device=l.device)
    if s["groups"] > 1:
        G = s["groups"]
        per = value.reshape(T, G, E // G)
        first, where = per.max(2)
        rank = first
        if s["best"] == 2 and E > G:
            rest = per.scatter(2, where[:, :, None], -math.inf).amax(2)
            rank = torch.where(rest > -math.inf, first + rest, first)
        # a group is kept when fewer than top_groups come before it
        g = torch.arange(G, device=l.device)
        ahead = (rank[:, None, :] > rank[:, :, None]) | ((rank[:, None, :] == rank[:, :, None]) & (g[None, :] < g[:, None]))
        open_ = (ahead.sum(2) < s["top_groups"]).repeat_interleave(E // G, 1)
    experts = []
    for _ in range(s["k"]):
        v = torch.where(open_, value, math.nan)
        most = torch.where(open_, value, -math.inf).amax(1, keepdim=True)
        e = torch.where(open_ & (v == most), index, E).amin(1)
        experts.append(e)
        open_[rows, e] = False
    return torch.stack(experts, 1), torch.where(torch.isneginf(l), 0.0, score)


def _exact_places(experts, E):
    chosen = torch.zeros((experts.shape[0], E), dtype=torch.int64, device=experts.device).scatter_(1, experts, 1)
    load = chosen.sum(0)
    start = load.cumsum(0) - load
    rank = chosen.cumsum(0) - chosen   # earlier tokens of the same expert
    return torch.gather(start[None] + rank, 1, experts), torch.cat([load.new_zeros(1), load.cumsum(0)])


def _exact_weights(experts, score, s):
    w = torch.gather(score, 1, experts)
    if s["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return s["scale"] * w


def _exact_scores(s):
    l = s["logits"].double()
    experts, score = _exact_choice(l, s["b"], s)
    positions, offsets = _exact_places(experts, s["E"])
    w = _exact_weights(experts, score, s)
    got = [experts.int(), w, offsets.int(), positions.int()]
    if s["grad"]:
        # through the weights to the scores, then through the scores to the logits
        d = s["dweights"].double() * s["scale"]
        if s["renormalize"]:
            total = torch.gather(score, 1, experts).sum(1, keepdim=True)
            d = torch.where(total > 0, (d - (d * w).sum(1, keepdim=True) / s["scale"]) / total, 0.0)
        ds = torch.zeros_like(l).scatter_(1, experts, d)
        got.append(ds * score * (1 - score) if s["score"] == "sigmoid" else score * (ds - (ds * score).sum(1, keepdim=True)))
    return got


def _exact_rounded(x):
    """Each block's values to the nearest code by distance, the even code among two as near."""
    T, K = x.shape
    x = x.double().reshape(-1, 32)
    most = x.abs().max(1, keepdim=True).values
    step = torch.where(most > 0, 2.0 ** (torch.floor(torch.log2(most)) - 2).clamp(-127, 127), 1.0)
    a = (x / step).abs()
    best = torch.zeros_like(a)
    for code in (2, 4, 6, 1, 3, 5, 7):   # even codes first: an odd one has to be nearer
        v = VALUES[code]
        best = torch.where((a - v).abs() < (a - best).abs(), v, best)
    return (torch.sign(x) * best * step).reshape(T, K)


def _exact_unpack(codes, scale):
    table = torch.tensor([(-1.0 if c & 8 else 1.0) * VALUES[c & 7] for c in range(16)], dtype=torch.float64, device=codes.device)
    out = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device=codes.device)
    out[..., 0::2] = table[(codes % 16).long()]
    out[..., 1::2] = table[(codes // 16).long()]
    for block in range(out.shape[-1] // 32):
        out[..., 32 * block:32 * block + 32] *= 2.0 ** (scale[block // 8, ..., block % 8].double()[..., None] - 127)
    return out


def _exact_ffn(s):
    l = s["logits"].double()
    sc = _ffn_scores(s)
    experts, score = _exact_choice(l, s["b"], sc)
    w = _exact_weights(experts, score, sc)
    x = _exact_rounded(s["x"])
    out = x.new_zeros((s["T"], s["H"]))
    for e in range(s["E"]):
        token, slot = torch.nonzero(experts == e, as_tuple=True)
        if len(token):
            y = x[token] @ _exact_unpack(s["w1"][e], s["s1"][:, e]).T
            h = _exact_rounded(y[:, :s["I"]] * torch.sigmoid(y[:, :s["I"]]) * y[:, s["I"]:])
            out.index_add_(0, token, w[token, slot, None] * (h @ _exact_unpack(s["w2"][e], s["s2"][:, e]).T))
    return out


def _exact_kept(x):
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], BLOCK8):
        b = x[:, lo:lo + BLOCK8]
        most = b.abs().max(1, keepdim=True).values
        out[:, lo:lo + BLOCK8] = torch.where(most > 0, torch.round(127 * b / most) * most / 127, 0.0)
    return out


def _exact_gate(s):
    I, at = s["I"], s["positions"].long()
    w = torch.empty(at.numel(), dtype=torch.float64, device=at.device)
    w[at] = s["weights"].double()
    w = w[:, None]
    gu, dh = s["gu"].double(), s["dh"].double()
    first = w * torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    g, u = _exact_kept(gu[:, :I]), _exact_kept(gu[:, I:])
    sig = torch.sigmoid(g)
    slope = sig + g * sig * (1 - sig)
    h = g * sig * u
    return [first, torch.cat([w * dh * u * slope, w * dh * g * sig], 1), w * h, (dh * h).sum(1)[at]]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "scores":
        return _exact_scores(s)
    if s["op"] == "quantize":
        return _exact_rounded(s["x"])
    if s["op"] == "product":
        if s["E"] == 0:
            return _exact_rounded(s["x"]) @ _exact_unpack(s["w"], s["ws"]).T
        out = torch.empty((s["M"], s["N"]), dtype=torch.float64, device="cuda")
        lo = 0
        for e, n in enumerate(s["counts"]):
            out[lo:lo + n] = _exact_unpack(s["x"][lo:lo + n], s["xs"][:, lo:lo + n]) @ _exact_unpack(s["w"][e], s["ws"][:, e]).T
            lo += n
        return out
    return _exact_ffn(s) if s["op"] == "ffn" else _exact_gate(s)


# ---- what a pass cannot do without ----------------------------------------------

def _busy(E, R):
    """Experts that get any of R rows spread evenly: their weights are read."""
    return E * (1 - (1 - 1 / E) ** R)


def _mx(n):
    """Bytes of n values: half a byte each and a byte for 32."""
    return n * 17 / 32


def work(case):
    if case["op"] == "scores":
        T, E, k = case["T"], case["E"], case["k"]
        b = T * E * 4 + (E * 4 if case["bias"] else 0) + T * k * 12 + (E + 1) * 4
        f = T * (E * 4 + 6 * k)
        if case["grad"]:   # the gradient writes every logit; a softmax over all reads them again, sigmoid the chosen
            b += T * E * 4 + T * k * 4
            f += T * k * 8 + (T * E * 4 if case["score"] == "softmax" and not case["renormalize"] else 0)
        return {"bytes": b, "flops": f}
    if case["op"] == "quantize":   # in, the codes out and in again, out
        n = case["T"] * case["K"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 2 * _mx(n) + 2 * n, "flops": 4 * n}
    if case["op"] == "product":
        M, N, K, E = case["M"], case["N"], case["K"], case["E"]
        weights = 1 if E == 0 else _busy(max(E - case["empty"], 1), M)
        b = (2 * M * K if E == 0 else _mx(M * K)) + weights * _mx(N * K) + M * N * (2 if case["out"] == "bf16" else 4)
        return {"bytes": b + (0 if E == 0 else (E + 1) * 4), "flops": 2 * M * N * K}
    if case["op"] == "ffn":
        T, E, k, H, I = (case[x] for x in ("T", "E", "k", "H", "I"))
        return {"bytes": T * E * 4 + E * 4 + 2 * T * H * 2 + _busy(E, T * k) * _mx(3 * I * H), "flops": 2 * T * k * 3 * I * H}
    T, k, I = case["T"], case["k"], case["I"]
    R, kept = T * k, 2 * case["I"] + 8 * -(-case["I"] // BLOCK8)
    # forward: 2I in, I and what is kept out; backward: what is kept and I in, 2I and I out
    return {"bytes": R * (4 * I + 2 * I + kept) + R * (kept + 2 * I + 4 * I + 2 * I) + 2 * T * k * 8 + T * k * 4, "flops": R * I * 30}
