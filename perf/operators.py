"""The operators of an expert layer around the grouped products, as they are
measured: what each call gets, what it returns and what it cannot do without.

Four operators, each reached through the package's own entry points:

* route     the router's selection: the k largest of E logits of each token,
            their softmax weights, and the order that groups the
            token-expert pairs by expert; for training also the gradient of
            the logits;
* rows      moving rows between the token order and the grouped order: the
            copy of each token's row to its k experts (dispatch) and the
            weighted sum of the k results (combine), each with its gradient;
* product   the matrix product in 8-bit integers with one scale per token and
            one per (expert, output channel): grouped by expert with ragged
            sizes, and dense from BF16 rows, which are quantised in the call;
* ffn       the three together as a serving step runs them: a gated
            feed-forward block of E experts in 8-bit integers, from BF16
            rows and router logits to BF16 rows.

With `own` false, run() computes the same from elementary torch operations in
FP32, rounded once at the end.  Sizes are those of the package's workloads
(E = 8 and 32 experts, d_model 2048, gate_up 1536, down 768, 16384 tokens on
256 experts, 131072 rows, the 4096 x 4096 projection), single tokens and
batches of a few, and odd sizes between them.
"""
import math

import torch

own = False

# the largest product of the listed cases: rows x output channels x reduction
MOST_WORK = 131072 * (2048 * 1536 + 768 * 2048)


def listed():
    return [
        # one token of a decoding step through the router of 256 experts
        {"name": "route_token", "op": "route", "T": 1, "E": 256, "k": 8, "renormalize": True, "grad": False, "padded": 0.0},
        # a prompt of odd length on 32 experts, weights from the softmax over all experts, an eighth of it padding
        {"name": "route_prompt", "op": "route", "T": 2039, "E": 32, "k": 2, "renormalize": False, "grad": False, "padded": 0.125},
        # a training step's 16384 tokens on 256 experts, forward and the logits' gradient
        {"name": "route_train", "op": "route", "T": 16384, "E": 256, "k": 8, "renormalize": True, "grad": True, "padded": 0.0},
        # the weighted sum at the end of a decoding step for 16 sequences
        {"name": "rows_decode", "op": "rows", "what": "combine", "T": 16, "k": 8, "H": 2048, "dtype": "bf16", "grad": False},
        # dispatch in FP32 rows of an odd batch, forward and gradient
        {"name": "rows_dispatch_odd", "op": "rows", "what": "dispatch", "T": 5003, "k": 2, "H": 776, "dtype": "fp32", "grad": True},
        # the weighted sum of a training step, forward and the gradients of rows and weights
        {"name": "rows_train", "op": "rows", "what": "combine", "T": 16384, "k": 8, "H": 2048, "dtype": "bf16", "grad": True},
        # one decoded token through the square projection, from BF16
        {"name": "product_token", "op": "product", "E": 0, "M": 1, "N": 4096, "K": 4096, "skew": 0.0, "empty": 0, "out": "bf16"},
        # 64 rows of a decoding step spread over 32 experts (gate_up)
        {"name": "product_decode", "op": "product", "E": 32, "M": 64, "N": 1536, "K": 2048, "skew": 0.0, "empty": 0, "out": "bf16"},
        # a Zipf-routed prompt on the down shape, two experts without rows, FP32 output
        {"name": "product_ragged", "op": "product", "E": 32, "M": 16411, "N": 2048, "K": 768, "skew": 1.2, "empty": 2, "out": "fp32"},
        # the gate_up product at its full size
        {"name": "product_full", "op": "product", "E": 8, "M": 131072, "N": 1536, "K": 2048, "skew": 0.0, "empty": 0, "out": "bf16"},
        # a decoding step of 8 sequences through the whole block
        {"name": "ffn_decode", "op": "ffn", "T": 8, "E": 32, "k": 4, "H": 2048, "I": 768},
        # 16384 prompt tokens through the whole block, 8 experts each
        {"name": "ffn_prompt", "op": "ffn", "T": 16384, "E": 32, "k": 8, "H": 2048, "I": 768},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "rows", "product", "ffn"])
    if op == "route":
        E = rng.choice([8, 32, 64, 100, 256])
        return {"op": op, "T": _log(rng, 1, 16384) | 1, "E": E, "k": rng.randint(1, 8), "renormalize": rng.random() < 0.7,
                "grad": rng.random() < 0.5, "padded": rng.choice([0.0, 0.2])}
    if op == "rows":
        return {"op": op, "what": rng.choice(["combine", "dispatch"]), "T": _log(rng, 1, 16000) | 1, "k": rng.randint(1, 8),
                "H": 8 * (2 * rng.randint(16, 127) + 1), "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "grad": rng.random() < 0.6}
    if op == "product":
        E = rng.choice([0, 1, 8, 32, 57])
        N, K = 8 * (2 * rng.randint(32, 200) + 1), 16 * (2 * rng.randint(8, 100) + 1)
        most = min(65536, MOST_WORK // (N * K))
        return {"op": op, "E": E, "M": _log(rng, 1, most) | 1, "N": N, "K": K, "skew": rng.choice([0.0, 1.2]),
                "empty": 2 if E > 8 else 0, "out": rng.choice(["bf16", "fp32"])}
    return {"op": op, "T": _log(rng, 1, 8000) | 1, "E": rng.choice([8, 32, 57]), "k": rng.randint(1, 8),
            "H": 16 * (2 * rng.randint(16, 63) + 1), "I": 16 * (2 * rng.randint(8, 23) + 1)}


# ---- inputs -------------------------------------------------------------------

def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _codes(g, *shape):
    """8-bit codes as quantising normal values gives them (the largest of a
    row of some thousand is about 3.7 standard deviations), and scales."""
    q = torch.randn(shape, generator=g, device="cuda").mul_(34).round_().clamp_(-127, 127).to(torch.int8)
    return q, torch.rand(shape[:-1], generator=g, device="cuda") * 0.001 + 0.0005


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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        s["logits"] = _logits(g, case)
        if case["grad"]:
            s["dweights"] = _normal(g, case["T"], case["k"])
    elif case["op"] == "rows":
        T, k, H = case["T"], case["k"], case["H"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # k distinct experts of 64 for each token, grouped by expert
        experts = torch.rand((T, 64), generator=g, device="cuda").argsort(1)[:, :k]
        s["positions"] = experts.flatten().argsort(stable=True).argsort().to(torch.int32).reshape(T, k)
        if case["what"] == "combine":
            s["weights"] = torch.softmax(_normal(g, T, k), 1)
            s["rows"] = _normal(g, T * k, H, dtype=dt)
            if case["grad"]:
                s["dout"] = _normal(g, T, H, dtype=dt)
        else:
            s["rows"] = _normal(g, T, H, dtype=dt)
            if case["grad"]:
                s["dout"] = _normal(g, T * k, H, dtype=dt)
    elif case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        if case["E"] == 0:
            s["x"] = _normal(g, M, K, dtype=torch.bfloat16)
            s["w"], s["ws"] = _codes(g, N, K)
        else:
            s["x"], s["xs"] = _codes(g, M, K)
            s["w"], s["ws"] = _codes(g, case["E"], N, K)
            counts = _counts(h, case["E"], M, case["skew"], case["empty"])
            s["counts"] = counts.tolist()
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32).cuda()
    else:
        s["logits"] = _logits(g, case)
        s["x"] = _normal(g, case["T"], case["H"], dtype=torch.bfloat16)
        s["w1"], s["s1"] = _codes(g, case["E"], 2 * case["I"], case["H"])
        s["w2"], s["s2"] = _codes(g, case["E"], case["H"], case["I"])
    return s


# ---- the plain form -------------------------------------------------------------

def _plain_route(logits, k, renormalize):
    top, experts = torch.sort(logits, dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k]
    most = top[:, :1]
    p = torch.exp(torch.where(most == -math.inf, -math.inf, top - most))
    total = (p if renormalize else torch.exp(torch.where(most == -math.inf, -math.inf, logits - most))).sum(1, keepdim=True)
    weights = p / torch.where(total == 0, 1.0, total)
    order = torch.sort(experts.reshape(-1), stable=True)[1]
    positions = torch.empty_like(order)
    positions[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.zeros(logits.shape[1] + 1, dtype=torch.int64, device=logits.device)
    offsets[1:] = torch.bincount(experts.reshape(-1), minlength=logits.shape[1]).cumsum(0)
    return (experts.to(torch.int32), weights, offsets.to(torch.int32), positions.reshape(experts.shape).to(torch.int32))


def _plain_route_grad(dweights, logits, experts, weights, renormalize):
    inner = (dweights * weights).sum(1, keepdim=True)
    at = experts.long()
    if renormalize:
        return torch.zeros_like(logits).scatter_(1, at, weights * (dweights - inner))
    most = logits.amax(1, keepdim=True)
    p = torch.exp(torch.where(most == -math.inf, -math.inf, logits - most))
    total = p.sum(1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    return p * (torch.zeros_like(logits).scatter_(1, at, dweights) - inner)


def _plain_rows(s):
    T, k, H = s["T"], s["k"], s["H"]
    at, rows = s["positions"].long(), s["rows"].float()
    if s["what"] == "dispatch":
        out = torch.empty((T * k, H), device=rows.device)
        out[at.reshape(-1)] = rows.repeat_interleave(k, 0)
        got = [out.to(s["rows"].dtype)]
        if s["grad"]:
            got.append(s["dout"].float()[at].sum(1).to(s["rows"].dtype))
        return got
    picked = rows[at]
    got = [(picked * s["weights"][:, :, None]).sum(1).to(s["rows"].dtype)]
    if s["grad"]:
        dout = s["dout"].float()[:, None, :]
        drows = torch.empty_like(rows)
        drows[at.reshape(-1)] = (s["weights"][:, :, None] * dout).reshape(T * k, H)
        got += [drows.to(s["rows"].dtype), (picked * dout).sum(2)]
    return got


def _plain_quantize(x):
    x = x.float()
    most = x.abs().amax(1, keepdim=True)
    return torch.round(x * 127 / torch.where(most == 0, 1.0, most)), most[:, 0] / 127


def _plain_grouped(x, xs, w, ws, counts):
    y = torch.cat([a @ b.float().T * c for a, b, c in zip(x.float().split(counts), w, ws[:, None, :])])
    return y * xs[:, None]


def _plain_ffn(s):
    experts, weights, offsets, positions = _plain_route(s["logits"], s["k"], True)
    counts = (offsets[1:] - offsets[:-1]).tolist()
    at = positions.long()
    x, xs = _plain_quantize(s["x"])
    token = torch.empty(at.numel(), dtype=torch.int64, device=at.device)
    token[at.reshape(-1)] = torch.arange(at.shape[0], device=at.device).repeat_interleave(at.shape[1])
    y = _plain_grouped(x[token], xs[token], s["w1"], s["s1"], counts)
    gate, up = y[:, :s["I"]], y[:, s["I"]:]
    h, hs = _plain_quantize(gate / (1 + torch.exp(-gate)) * up)
    y = _plain_grouped(h, hs, s["w2"], s["s2"], counts)
    return (y[at] * weights[:, :, None]).sum(1).to(torch.bfloat16)


def _plain(s):
    if s["op"] == "route":
        got = _plain_route(s["logits"], s["k"], s["renormalize"])
        if s["grad"]:
            got += (_plain_route_grad(s["dweights"], s["logits"], got[0], got[1], s["renormalize"]),)
        return got
    if s["op"] == "rows":
        return _plain_rows(s)
    if s["op"] == "product":
        dt = torch.bfloat16 if s["out"] == "bf16" else torch.float32
        if s["E"] == 0:
            x, xs = _plain_quantize(s["x"])
            return (x @ s["w"].float().T * s["ws"] * xs[:, None]).to(dt)
        return _plain_grouped(s["x"], s["xs"], s["w"], s["ws"], s["counts"]).to(dt)
    return _plain_ffn(s)


# ---- the framework's operators -------------------------------------------------

def _own(s):
    import dense_ragged_grouped_amd as drgg
    from dense_ragged_grouped_amd import moe
    if s["op"] == "route":
        r = drgg.moe_route(s["logits"], s["k"], renormalize=s["renormalize"])
        got = (r.experts, r.weights, r.group_offsets, r.positions)
        if s["grad"]:
            got += (drgg.moe_route_grad(s["dweights"], s["logits"], r.experts, r.weights, renormalize=s["renormalize"]),)
        return got
    if s["op"] == "rows":
        if s["what"] == "dispatch":
            got = [drgg.moe_dispatch(s["rows"], s["positions"])]
            if s["grad"]:
                got.append(drgg.moe_combine(s["dout"], s["positions"]))
            return got
        got = [drgg.moe_combine(s["rows"], s["positions"], s["weights"])]
        if s["grad"]:
            got += drgg.moe_combine_grad(s["dout"], s["rows"], s["positions"], s["weights"])
        return got
    if s["op"] == "product":
        dt = torch.bfloat16 if s["out"] == "bf16" else torch.float32
        if s["E"] == 0:
            x, xs = drgg.quantize_int8(s["x"])
            return drgg.gemm_int8(x, xs, s["w"], s["ws"], out_dtype=dt)
        return drgg.grouped_gemm_int8(s["x"], s["xs"], s["w"], s["ws"], s["offsets"], out_dtype=dt)
    return moe.ffn_int8(s["x"], s["logits"], s["w1"], s["s1"], s["w2"], s["s2"], s["k"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- the same from the definitions, in 64 bits ------------------------------------

def _exact_choice(logits, k):
    """The k experts of each token by taking the largest logit k times (the
    lowest index among equals), and each pair's place in the grouped order."""
    T, E = logits.shape
    left, chosen = logits.clone(), torch.zeros((T, E), dtype=torch.bool, device=logits.device)
    index = torch.arange(E, device=logits.device)
    experts = []
    for _ in range(k):
        free = left.masked_fill(chosen, math.nan)
        best = torch.where(chosen, -math.inf, free).amax(1, keepdim=True)
        e = torch.where((free == best) & ~chosen, index, E).amin(1)
        experts.append(e)
        chosen[torch.arange(T, device=e.device), e] = True
    experts = torch.stack(experts, 1)
    load = chosen.sum(0)
    start = load.cumsum(0) - load
    rank = chosen.long().cumsum(0) - chosen.long()   # earlier tokens of the same expert
    positions = torch.gather(start[None] + rank, 1, experts)
    return experts, positions, load


def _exact_softmax(v):
    most = v.max(1, keepdim=True).values
    p = torch.exp(v - torch.where(torch.isinf(most), 0.0, most))
    total = p.sum(1, keepdim=True)
    return torch.where(total > 0, p / total, 0.0)


def _exact_product(x, xs, w, ws):
    return (x.double() @ w.double().T) * xs.double()[:, None] * ws.double()[None, :]


def _exact_codes(x):
    x = x.double()
    most = x.abs().max(1, keepdim=True).values
    return torch.where(most > 0, torch.round(127 * x / most), 0.0), most[:, 0] / 127


def _exact_route(s):
    logits = s["logits"].double()
    experts, positions, load = _exact_choice(logits, s["k"])
    p = _exact_softmax(torch.gather(logits, 1, experts) if s["renormalize"] else logits)
    w = p if s["renormalize"] else torch.gather(p, 1, experts)
    offsets = torch.cat([load.new_zeros(1), load.cumsum(0)])
    got = [experts.int(), w, offsets.int(), positions.int()]
    if s["grad"]:
        d = s["dweights"].double()
        full = p.new_zeros(logits.shape)
        if s["renormalize"]:
            full.scatter_(1, experts, p * d - p * (p * d).sum(1, keepdim=True))
        else:
            up = torch.zeros_like(p).scatter_(1, experts, d)
            full = p * up - p * (p * up).sum(1, keepdim=True)
        got.append(full)
    return got


def _exact_rows(s):
    T, k, H = s["T"], s["k"], s["H"]
    at = s["positions"].long()
    rows = s["rows"].double()
    if s["what"] == "dispatch":
        source = torch.empty(T * k, dtype=torch.int64, device=at.device)
        source[at.reshape(-1)] = torch.arange(T * k, device=at.device) // k
        got = [rows[source]]
        if s["grad"]:
            got.append(torch.zeros_like(rows).index_add_(0, source, s["dout"].double()))
        return got
    w = s["weights"].double()
    out = rows.new_zeros((T, H))
    for j in range(k):
        out += w[:, j, None] * rows[at[:, j]]
    got = [out]
    if s["grad"]:
        d = s["dout"].double()
        drows, dw = torch.empty_like(rows), torch.empty_like(w)
        for j in range(k):
            drows[at[:, j]] = w[:, j, None] * d
            dw[:, j] = (d * rows[at[:, j]]).sum(1)
        got += [drows, dw]
    return got


def _exact_ffn(s):
    experts, positions, load = _exact_choice(s["logits"].double(), s["k"])
    w = _exact_softmax(torch.gather(s["logits"].double(), 1, experts))
    x, xs = _exact_codes(s["x"])
    out = x.new_zeros((s["T"], s["H"]))
    for e in range(s["E"]):
        token, slot = torch.nonzero(experts == e, as_tuple=True)
        y = _exact_product(x[token], xs[token], s["w1"][e], s["s1"][e])
        h, hs = _exact_codes(y[:, :s["I"]] * torch.sigmoid(y[:, :s["I"]]) * y[:, s["I"]:]) if len(token) else (y[:, :s["I"]], y[:, 0])
        out.index_add_(0, token, w[token, slot, None] * _exact_product(h, hs, s["w2"][e], s["s2"][e]))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "route":
        return _exact_route(s)
    if s["op"] == "rows":
        return _exact_rows(s)
    if s["op"] == "product":
        if s["E"] == 0:
            return _exact_product(*_exact_codes(s["x"]), s["w"], s["ws"])
        out = torch.empty((s["M"], s["N"]), dtype=torch.float64, device="cuda")
        lo = 0
        for e, n in enumerate(s["counts"]):
            out[lo:lo + n] = _exact_product(s["x"][lo:lo + n], s["xs"][lo:lo + n], s["w"][e], s["ws"][e])
            lo += n
        return out
    return _exact_ffn(s)


# ---- what a pass cannot do without ----------------------------------------------

def _busy(E, R):
    """Experts that get any of R rows spread evenly: their weights are read."""
    return E * (1 - (1 - 1 / E) ** R)


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b = T * E * 4 + T * k * 12 + (E + 1) * 4
        f = T * (E * (1 if case["renormalize"] else 3) + 6 * k)
        if case["grad"]:   # the gradient writes every logit; a softmax over all reads them again
            b += T * E * 4 + T * k * 4
            f += T * (E if case["renormalize"] else 4 * E) + T * k * 4
        return {"bytes": b, "flops": f}
    if case["op"] == "rows":
        T, k, H = case["T"], case["k"], case["H"]
        row = H * (2 if case["dtype"] == "bf16" else 4)
        b, f = T * (k + 1) * row + T * k * 4, T * k * H
        if case["what"] == "combine":
            b, f = b + T * k * 4, 2 * f
        if case["grad"]:   # dispatch: k rows in, one out; combine: one in, k out, and the weights' gradient
            b += T * (k + 1) * row + (T * k * 4 if case["what"] == "combine" else 0)
            f *= 2
        return {"bytes": b, "flops": f}
    if case["op"] == "product":
        M, N, K, E = case["M"], case["N"], case["K"], case["E"]
        weights = 1 if E == 0 else _busy(max(E - case["empty"], 1), M)
        b = M * K * (2 if E == 0 else 1) + weights * N * (K + 4) + M * N * (2 if case["out"] == "bf16" else 4)
        return {"bytes": b + (0 if E == 0 else M * 4 + (E + 1) * 4), "flops": 2 * M * N * K}
    T, E, k, H, I = (case[x] for x in ("T", "E", "k", "H", "I"))
    return {"bytes": T * E * 4 + 2 * T * H * 2 + _busy(E, T * k) * 3 * I * H, "flops": 2 * T * k * 3 * I * H}
