"""The selection by scores and its gradient on the GPU, against plain
implementations in 64 bits (NumPy).

Tolerances, u = 2^-24:
* The choice is that of 64-bit values: equal, also where values differ by less
  than FP32 can hold.
* A sigmoid weight: the exponentials within 2 u of themselves, 1 + e and the
  quotient one rounding each; renormalised, the exponent x - m is rounded (|x -
  m| u of the term) and the sum of k <= 64 terms in a row of lanes is within 8 u;
  quotient and scale 2 u.  Together below (far + 20) u, doubled.
* A softmax weight: (far + V + 20) u, doubled, with V <= 64 terms added in a
  lane before the tree over lanes.
* The gradient: 1 - s is within 6 u of itself, sums and products of k (or E)
  factors with the weights' error on each.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module")
def drgg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as d
    import dense_ragged_grouped_amd.moe  # noqa: F401
    return d


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def scores64(logits, kind):
    l = logits.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            e = np.exp(-np.abs(l))
            return np.where(l < 0, e / (1 + e), 1 / (1 + e))
        most = l.max(1, keepdims=True) if l.size else l[:, :1]
        p = np.exp(l - np.where(np.isneginf(most), 0, most))
        total = p.sum(1, keepdims=True)
        return p / np.where(total == 0, 1, total)


def order(v):
    """Indices by value decreasing, NaN first, then by index."""
    nan = np.isnan(v)
    return sorted(range(len(v)), key=lambda e: (not nan[e], -(0.0 if nan[e] else v[e]), e))


def choose(logits, bias, c, k):
    """(experts [T, k], scores, masked) by Python's sorts of 64-bit values."""
    T, E = logits.shape
    s = scores64(logits, c["score"])
    b = np.zeros(E, np.float32) if bias is None else bias
    with np.errstate(invalid="ignore"):
        masked = np.isneginf(logits) | np.isneginf(b)[None]
        v = np.where(masked, -np.inf, s + b.astype(np.float64))
    if bias is None and c["groups"] == 1:
        v = logits.astype(np.float64)
    size = E // c["groups"]
    experts = np.empty((T, k), dtype=np.int64)
    for t in range(T):
        open_ = range(E)
        if c["groups"] > 1:
            rank = np.empty(c["groups"])
            for g in range(c["groups"]):
                part = v[t, g * size:(g + 1) * size]
                best = [part[i] for i in order(part)[:c["best"]]]
                rank[g] = best[0] if len(best) == 1 or np.isneginf(best[1]) else best[0] + best[1]
            kept = set(order(rank)[:c["top_groups"]])
            open_ = [e for e in range(E) if e // size in kept]
        open_ = np.array(open_)
        experts[t] = open_[order(v[t, open_])[:k]]
    return experts, s, masked


def weights64(experts, s, masked, logits, c):
    w = np.where(masked, 0.0, s)
    w = np.take_along_axis(w, experts, 1)
    if c["renormalize"]:   # a ratio: of logarithms, which hold scores below any range
        l = logits.astype(np.float64)
        with np.errstate(invalid="ignore"):
            log = l if c["score"] == "softmax" else np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
        log = np.take_along_axis(np.where(masked, -np.inf, log), experts, 1)
        most = log.max(1, keepdims=True) if log.size else log[:, :1]
        w = np.exp(log - np.where(np.isneginf(most), 0, most))
        total = w.sum(1, keepdims=True)
        w = w / np.where(total == 0, 1, total)
    return c["scale"] * w


def places(experts, E):
    T, k = experts.shape
    flat = experts.reshape(-1)
    at = np.argsort(flat, kind="stable")
    positions = np.empty(T * k, dtype=np.int64)
    positions[at] = np.arange(T * k)
    return positions.reshape(T, k), np.searchsorted(flat[at], np.arange(E + 1))


def config(score="sigmoid", groups=1, top_groups=1, best=2, renormalize=True, scale=1.0):
    return dict(score=score, groups=groups, top_groups=top_groups, best=best, renormalize=renormalize, scale=scale)


def make(kind, T, E, seed):
    """(logits, bias or None)"""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, E)).astype(np.float32)
    bias = (np.round(rng.standard_normal(E) * 30) * 0.001).astype(np.float32)
    if kind == "plain":
        bias = None
    elif kind == "ties":   # none negative: sums of two tie only where their terms do
        x, bias = rng.integers(0, 4, (T, E)).astype(np.float32), None
        x[x == 0] *= np.where(rng.random((x == 0).sum()) < 0.5, -1, 1)   # both zeros
    elif kind == "close":   # all values within some 2^-25 of each other
        x[:] = x[:1] if T else x
        bias = (1 - scores64(x[:1], "sigmoid")[0]).astype(np.float32) if T else bias
    elif kind == "masked":
        x[rng.random((T, E)) < 0.8] = -np.inf
        x[::3] = -np.inf
        bias[rng.random(E) < 0.2] = -np.inf
    elif kind == "lowest":
        x[rng.random((T, E)) < 0.8] = np.finfo(np.float32).min
        x[::3] = np.finfo(np.float32).min
    elif kind == "wide":
        x *= 30
    elif kind == "low":   # every score below FP32's range
        x = x * 5 - 300
    return x, bias


SHAPES = [(0, 8, 2, 1, 1), (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (2, 3, 3, 1, 1), (63, 8, 2, 4, 1), (64, 100, 5, 4, 3),
          (65, 32, 4, 8, 2), (130, 257, 8, 1, 1), (193, 60, 7, 5, 3), (67, 511, 7, 7, 2), (70, 1024, 64, 64, 5),
          (131, 1000, 6, 8, 4), (515, 64, 8, 16, 16), (66, 24, 17, 2, 2)]


@pytest.mark.parametrize("kind", ["bias", "plain", "ties", "close", "masked", "lowest", "wide", "low"])
@pytest.mark.parametrize("T,E,k,groups,top", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_choice_and_weights(drgg, T, E, k, groups, top, score, kind):
    if kind == "low" and score == "softmax":
        pytest.skip("a softmax does not see a shift")
    logits, bias = make(kind, T, E, T + E + k)
    for best in ((1, 2) if groups > 1 else (2,)):
        for renormalize, scale in ((True, 2.5), (False, 1.0)):
            c = config(score, groups, top, best, renormalize, scale)
            r = drgg.moe_route_scores(dev(logits), k, drgg.Scoring(**c, bias=None if bias is None else dev(bias)))
            experts, s, masked = choose(logits, bias, c, k)
            positions, offsets = places(experts, E)
            assert np.array_equal(host(r.experts), experts), (best, renormalize)
            assert np.array_equal(host(r.positions), positions)
            assert np.array_equal(host(r.group_offsets), offsets)
            assert np.array_equal(host(r.tokens)[positions.reshape(-1)], np.repeat(np.arange(T), k))
            w, want = host(r.weights), weights64(experts, s, masked, logits, c)
            with np.errstate(invalid="ignore"):
                x = np.take_along_axis(logits.astype(np.float64), experts, 1)
                if score == "sigmoid":
                    x = np.minimum(x, 0)
                far = np.abs(x - (logits.max(1, keepdims=True) if score == "softmax" and T else x.max(1, keepdims=True)))
            far = np.where(np.isfinite(far), far, 0)
            tol = 2 * (far + 20 + (64 if score == "softmax" else 0)) * U
            assert np.all(np.abs(w - want) <= tol * want + 2.0 ** -126)
            assert not w[np.take_along_axis(masked, experts, 1)].any()


def test_close_values_are_decided_in_64_bits(drgg):
    """The kind of input above in which FP32 values do not decide: their order differs from the 64-bit one's."""
    logits, bias = make("close", 1, 256, 0)
    v64 = scores64(logits, "sigmoid")[0] + bias.astype(np.float64)
    v32 = (scores64(logits, "sigmoid")[0].astype(np.float32) + bias).astype(np.float64)
    assert order(v64)[:8] != order(v32)[:8] and len(np.unique(v64)) == 256


@pytest.mark.parametrize("T,E,k", [(32769, 130, 2), (70001, 6, 1), (33000, 320, 3)])
def test_many_tokens(drgg, T, E, k):
    """More than 512 blocks of tokens: the counts go through the scan."""
    rng = np.random.default_rng(T)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    bias = rng.standard_normal(E).astype(np.float32)
    r = drgg.moe_route_scores(dev(logits), k, drgg.Scoring(bias=dev(bias)))
    v = scores64(logits, "sigmoid") + bias.astype(np.float64)
    experts = np.argsort(-v, axis=1, kind="stable")[:, :k]
    positions, offsets = places(experts, E)
    assert np.array_equal(host(r.experts), experts)
    assert np.array_equal(host(r.positions), positions) and np.array_equal(host(r.group_offsets), offsets)


def test_without_bias_and_groups_as_moe_route(drgg):
    """Softmax scores, one group, no bias: moe_route's results, bitwise its integers and, renormalised, its weights
    to rounding; NaN and infinities among the logits too."""
    rng = np.random.default_rng(4)
    logits = rng.standard_normal((300, 40)).astype(np.float32)
    logits[rng.random(logits.shape) < 0.1] = -np.inf
    logits[rng.random(logits.shape) < 0.005] = np.nan
    logits[rng.random(logits.shape) < 0.005] = np.inf
    a = drgg.moe_route(dev(logits), 5)
    b = drgg.moe_route_scores(dev(logits), 5, drgg.Scoring("softmax"))
    for x, y in ((a.experts, b.experts), (a.positions, b.positions), (a.group_offsets, b.group_offsets), (a.tokens, b.tokens)):
        assert torch.equal(x, y)
    fine = np.isfinite(logits).any(1) & ~(np.isnan(logits) | np.isposinf(logits)).any(1)
    assert np.allclose(host(a.weights)[fine], host(b.weights)[fine], rtol=100 * U, atol=0)


def test_nan_and_infinities(drgg):
    """A NaN value comes first with a NaN weight; an infinite logit has the score 1; an infinite bias decides; a
    softmax over NaN or infinity is NaN at every expert that is not masked."""
    nan, inf = np.nan, np.inf
    x = np.array([[0, nan, 1, -inf, 2, 3], [inf, 0, 1, 2, -inf, 3]], dtype=np.float32)
    r = drgg.moe_route_scores(dev(x), 3, drgg.Scoring("sigmoid", renormalize=False))
    assert host(r.experts).tolist() == [[1, 5, 4], [0, 5, 3]]
    w = host(r.weights)
    assert np.isnan(w[0, 0]) and np.isfinite(w[0, 1:]).all() and w[1, 0] == 1
    bias = np.array([0, 0, inf, 0, 0, -inf], dtype=np.float32)
    r = drgg.moe_route_scores(dev(x), 6, drgg.Scoring("sigmoid", bias=dev(bias), renormalize=False))
    assert host(r.experts).tolist() == [[1, 2, 4, 0, 3, 5], [2, 0, 3, 1, 4, 5]]
    assert host(r.weights)[0, 4:].tolist() == [0, 0] and host(r.weights)[1, 4:].tolist() == [0, 0]
    r = drgg.moe_route_scores(dev(x), 6, drgg.Scoring("softmax", bias=dev(np.zeros(6, np.float32))))
    assert host(r.experts).tolist() == [[0, 1, 2, 4, 5, 3], [0, 1, 2, 3, 5, 4]]
    assert np.isnan(host(r.weights)[:, :5]).all() and not host(r.weights)[:, 5].any()


# ---- gradient ------------------------------------------------------------------

def grad64(dw, s, masked, experts, c):
    """Through the weights to the scores, then to the logits."""
    T, E = s.shape
    s = np.where(masked, 0.0, s)
    chosen = np.take_along_axis(s, experts, 1)
    d = c["scale"] * np.where(chosen == 0, 0, dw)
    if c["renormalize"]:
        total = chosen.sum(1, keepdims=True)
        total = np.where(total == 0, 1, total)
        d = np.where(chosen == 0, 0, (d - (d * chosen).sum(1, keepdims=True) / total) / total)
    ds = np.zeros((T, E))
    np.put_along_axis(ds, experts, d, 1)
    if c["score"] == "sigmoid":
        return ds * s * (1 - s)
    # renormalised, ds and s are orthogonal
    return s * ds if c["renormalize"] else s * (ds - (ds * s).sum(1, keepdims=True))


@pytest.mark.parametrize("kind", ["bias", "masked", "wide"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 9, 3), (64, 256, 8), (33, 1000, 40), (130, 30, 17)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient(drgg, T, E, k, score, renormalize, kind):
    logits, bias = make(kind, T, E, T + E)
    c = config(score, renormalize=renormalize, scale=2.5)
    sc = drgg.Scoring(**c, bias=dev(bias))
    r = drgg.moe_route_scores(dev(logits), k, sc)
    experts = host(r.experts)
    s = scores64(logits, score)
    masked = np.isneginf(logits) | np.isneginf(bias)[None] & (score == "sigmoid" or renormalize)
    dw = np.random.default_rng(1).standard_normal((T, k)).astype(np.float32)
    got = dw.copy()
    got[host(r.weights) == 0] = np.nan   # not used
    got = host(drgg.moe_route_scores_grad(dev(got), dev(logits), r.experts, r.weights, sc))
    if score == "softmax" and not renormalize and np.isneginf(bias).any():
        # a bias of -inf takes its expert out of the choice, not out of the softmax
        gone = np.isneginf(bias)[None] | np.isneginf(logits)
        d = np.where(np.take_along_axis(gone, experts, 1), 0, dw)
        want = grad64(d, s, np.isneginf(logits), experts, c)
    else:
        want = grad64(dw.astype(np.float64), s, masked, experts, c)
    with np.errstate(invalid="ignore"):
        far = np.abs(logits - logits.max(1, keepdims=True)).astype(np.float64)
    far = np.where(np.isfinite(far), far, 0)
    w = host(r.weights)
    reach = (np.abs(dw) * (w > 0)).max(1, keepdims=True) + np.abs(w * dw).sum(1, keepdims=True) / c["scale"]
    if score == "softmax" and not renormalize:
        size = c["scale"] * np.where(np.isneginf(logits), 0, s) * reach
    else:
        size = np.zeros((T, E))
        np.put_along_axis(size, experts, w * reach, 1)
    # a weight underflows before its gradient does, so what is below FP32's range is left out
    assert np.all(np.abs(got - want) <= 8 * (far + 100 + k) * U * size + 2.0 ** -120)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(drgg, score, renormalize):
    T, E, k = 6, 12, 4
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    c = config(score, groups=3, top_groups=2, renormalize=renormalize, scale=1.7)
    x = dev(logits).requires_grad_()
    from dense_ragged_grouped_amd import moe
    r = moe.route_scores(x, k, drgg.Scoring(**c))
    dw = rng.standard_normal((T, k)).astype(np.float32)
    (r.weights * dev(dw)).sum().backward()
    experts = host(r.experts)

    def loss(l):
        return (weights64(experts, scores64(l, score), np.zeros((T, E), bool), l, c) * dw).sum()
    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = logits.astype(np.float64), logits.astype(np.float64)
            up[t, e] += h
            down[t, e] -= h
            # central differences: h^2 / 6 of a third derivative below 20, and rounding 1e-16 / h
            assert abs((loss(up) - loss(down)) / (2 * h) - float(x.grad[t, e])) < 1e-6


def test_second_derivative_raises(drgg):
    from dense_ragged_grouped_amd import moe
    x = torch.randn(4, 8, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(moe.route_scores(x, 2).weights.pow(2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()


# ---- calls ---------------------------------------------------------------------

def test_refusals(drgg):
    x = torch.randn(4, 12, device="cuda")
    S = drgg.Scoring
    for bad, error in ((S("relu"), ValueError), (S(groups=5), drgg.DrggError), (S(groups=3, top_groups=4), drgg.DrggError),
                       (S(groups=0), drgg.DrggError), (S(best=3), drgg.DrggError), (S(scale=0.0), drgg.DrggError),
                       (S(scale=float("nan")), drgg.DrggError), (S(scale=float("inf")), drgg.DrggError),
                       (S(groups=6, top_groups=1), drgg.DrggError),   # two experts, k = 3
                       (S(bias=torch.zeros(11, device="cuda")), ValueError), (S(bias=torch.zeros(12)), TypeError),
                       (S(bias=torch.zeros(12, device="cuda", dtype=torch.float64)), TypeError),
                       (S(bias=torch.zeros(24, device="cuda")[::2]), ValueError)):
        with pytest.raises(error):
            drgg.moe_route_scores(x, 3, bad)


def test_captured_and_replayed(drgg):
    """Two graphs of the selection and its gradient, replayed in turn on changing logits beside eager calls."""
    E, k = 64, 4
    bias = torch.randn(E, device="cuda") * 0.01
    sc = drgg.Scoring(bias=bias, groups=8, top_groups=3)
    made = []
    for T in (70, 200):
        x, dw = torch.randn(T, E, device="cuda"), torch.randn(T, k, device="cuda")

        def step(x=x, dw=dw):
            r = drgg.moe_route_scores(x, k, sc)
            return (*r, drgg.moe_route_scores_grad(dw, x, r.experts, r.weights, sc))
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        made.append((x, step, graph, out))
    for i in range(3):
        for x, step, graph, out in made:
            x.copy_(torch.randn_like(x))
            graph.replay()
            for a, b in zip(out, step()):
                assert torch.equal(a, b)


def test_on_another_stream(drgg):
    x, bias = torch.randn(130, 32, device="cuda"), torch.randn(32, device="cuda")
    sc = drgg.Scoring(bias=bias)
    want = drgg.moe_route_scores(x, 4, sc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = drgg.moe_route_scores(x, 4, sc, stream=side)
    dw = torch.ones(130, 4, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    grad = drgg.moe_route_scores_grad(dw, x, got.experts, got.weights, sc, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert torch.equal(grad, drgg.moe_route_scores_grad(dw, x, want.experts, want.weights, sc))


def test_large_biases(drgg):
    """Sums of two biases beyond FP32's range are still compared as 64-bit values."""
    x = torch.zeros(5, 16, device="cuda")
    bias = torch.full((16,), -3e38)
    bias[[0, 1, 8, 9]] = torch.tensor([3.1e38, 2.0e38, 3.0e38, 3.0e38])
    r = drgg.moe_route_scores(x, 3, drgg.Scoring(bias=bias.cuda(), groups=2, top_groups=1))
    assert host(r.experts).tolist() == [[8, 9, 10]] * 5


def test_int8_block_by_scores(drgg):
    """The 8-bit serving block with a Scoring that is moe_route's selection: the one call's result."""
    from dense_ragged_grouped_amd import moe
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    X = torch.randn(70, 64, generator=g, device="cuda").bfloat16()
    logits = torch.randn(70, 8, generator=g, device="cuda")
    w = (*moe.quantize_weights(torch.randn(8, 96, 64, generator=g, device="cuda")),
         *moe.quantize_weights(torch.randn(8, 64, 48, generator=g, device="cuda")))
    assert torch.equal(drgg.moe_route(logits, 2).weights, drgg.moe_route_scores(logits, 2, drgg.Scoring("softmax")).weights)
    assert torch.equal(moe.ffn_int8(X, logits, *w, 2), moe.ffn_int8(X, logits, *w, 2, scoring=drgg.Scoring("softmax")))
    sc = drgg.Scoring(bias=torch.linspace(-1, 1, 8, device="cuda"), scale=2.0)
    r = drgg.moe_route_scores(logits, 2, sc)
    q, s = drgg.quantize_int8(X)
    h = drgg.grouped_gemm_int8(q, s, w[0], w[1], r.group_offsets, gated=True, rows=r.tokens, out_dtype=torch.float32)
    y = drgg.grouped_gemm_int8(*drgg.quantize_int8(h), w[2], w[3], r.group_offsets)
    assert torch.equal(moe.ffn_int8(X, logits, *w, 2, scoring=sc), drgg.moe_combine(y, r.positions, r.weights))
