"""The gated activation kept in 8 bits, its backward pass and the training block
on them, on the GPU, against plain implementations in 64 bits (NumPy).

Tolerances, u = 2^-24:
* Codes and scales: equal (127 x / m of BF16 values is a half only where it is
  one exactly, and otherwise at least 2^-9 from it).
* silu(g) u: (|g| + 6) u for the sigmoid (its exponent's rounding, exponential,
  sum, reciprocal) and a rounding for each product: (4 |g| + 16) u, and 0 for
  the value below g = -87; then half a step of BF16.
* The gradient at the kept values: scale * code is rounded once, which moves
  s (1 + g (1 - s)) by at most |g| u / 2, beside (4 |g| + 32) u of its terms.
* dweights: I roundings in any order on top of the terms' own.
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
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def half_step(v):
    return 2.0 ** -8 * np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))))


def sigmoid64(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g))


def kept64(x):
    """(codes, scales) of a half [R, I]."""
    R, I = x.shape
    codes, scales = np.zeros((R, I), np.int8), np.zeros((R, -(-I // 128)), np.float32)
    for b in range(scales.shape[1]):
        v = x[:, 128 * b:128 * b + 128]
        bad = ~np.isfinite(v).all(1)
        v = np.where(bad[:, None], 0, v)
        m = np.abs(v).max(1)
        codes[:, 128 * b:128 * b + 128] = np.rint(127 * v / np.where(m == 0, 1, m)[:, None])
        scales[:, b] = np.where(bad, np.nan, (m.astype(np.float32) / np.float32(127)))
    return codes, scales


def make(T, k, I, kind, seed):
    rng = np.random.default_rng(seed)
    R = T * k
    gu = rng.standard_normal((R, 2 * I)).astype(np.float32)
    if kind == "wide":
        gu *= np.exp2(rng.integers(-20, 8, (R, 2 * I))).astype(np.float32)
    elif kind == "edges":
        gu[::4] = 0
        gu[1::4, : I // 2] *= np.float32(1e37)
        gu[2::4] *= np.float32(1e-39)
    weights = rng.random((T, k)).astype(np.float32)
    weights[rng.random((T, k)) < 0.1] = 0
    positions = rng.permutation(R).astype(np.int32).reshape(T, k)
    dh = rng.standard_normal((R, I)).astype(np.float32)
    return dev(gu).bfloat16(), dev(positions), dev(weights), dev(dh).bfloat16()


SHAPES = [(0, 2, 16), (1, 1, 8), (3, 2, 24), (5, 3, 128), (17, 1, 136), (33, 8, 768), (70, 2, 1288), (9, 64, 104), (4, 2, 2056),
          (2, 1, 5000)]


def row_weights(positions, weights):
    w = np.zeros(positions.numel())
    w[host(positions).reshape(-1)] = host(weights).reshape(-1)
    return w[:, None]


@pytest.mark.parametrize("kind", ["normal", "wide", "edges"])
@pytest.mark.parametrize("T,k,I", SHAPES)
def test_forward(drgg, T, k, I, kind):
    GU, positions, weights, _ = make(T, k, I, kind, T + I)
    h, codes, scale = drgg.moe_gate_int8(GU, positions, weights)
    gu, w = host(GU), row_weights(positions, weights)
    g, u = gu[:, :I], gu[:, I:]
    B = -(-I // 128)
    for half, lo, at in ((g, 0, 0), (u, I, B)):
        q, s = kept64(half)
        assert np.array_equal(host(codes)[:, lo:lo + I], q)
        assert np.array_equal(scale.cpu().numpy()[:, at:at + B], s)
    want = w * (g * sigmoid64(g)) * u
    tol = half_step(want) + (4 * np.abs(g) + 16) * U * np.abs(want)
    tol = np.where(g < -87, tol + np.abs(want), tol)
    got = host(h)
    fine = np.abs(want) < 2.0 ** 127
    assert np.all((np.abs(got - want) <= tol) | ~fine)
    assert not got[(w == 0).ravel()].any()


def grads64(dh, codes, scale, w, I):
    B = -(-I // 128)
    g = codes[:, :I] * np.repeat(scale[:, :B], 128, 1)[:, :I]
    u = codes[:, I:] * np.repeat(scale[:, B:], 128, 1)[:, :I]
    s = sigmoid64(g)
    act = g * s * u
    return g, u, s, act, w * dh * u * s * (1 + g * (1 - s)), w * dh * g * s


@pytest.mark.parametrize("kind", ["normal", "wide"])
@pytest.mark.parametrize("T,k,I", SHAPES)
def test_backward(drgg, T, k, I, kind):
    GU, positions, weights, dh = make(T, k, I, kind, T + I + 1)
    _, codes, scale = drgg.moe_gate_int8(GU, positions, weights)
    dGU, h, dw = drgg.moe_gate_int8_grad(dh, codes, scale, positions, weights)
    d, w = host(dh), row_weights(positions, weights)
    g, u, s, act, dg, du = grads64(d, host(codes).astype(np.float64), host(scale), w, I)
    rel = (4 * np.abs(g) + 32) * U
    low = np.where(g < -87, 1.0, 0.0)   # the sigmoid is 0 there
    terms = np.abs(w * d * u) * (s + np.abs(g) * s)
    got = host(dGU)
    assert np.all(np.abs(got[:, :I] - dg) <= half_step(dg) + (rel + low) * terms)
    assert np.all(np.abs(got[:, I:] - du) <= half_step(du) + (rel + low) * np.abs(w * d * g * s))
    assert np.all(np.abs(host(h) - w * act) <= half_step(w * act) + (rel + low) * np.abs(w * act))
    want = (d * act).sum(1)
    tol = ((I * U + rel + low) * np.abs(d * act)).sum(1)
    at = host(positions)
    assert np.all(np.abs(host(dw) - want[at]) <= tol[at] + 2.0 ** -126)
    assert not got[(w == 0).ravel()].any()


def test_backward_against_differences(drgg):
    """Of the forward formula in 64 bits at the kept values; BF16 results are within 2^-8 of their value."""
    T, k, I = 3, 2, 40
    GU, positions, weights, dh = make(T, k, I, "normal", 0)
    weights = weights + 0.1
    _, codes, scale = drgg.moe_gate_int8(GU, positions, weights)
    dGU, _, dw = (host(t) for t in drgg.moe_gate_int8_grad(dh, codes, scale, positions, weights))
    d, wr, q = host(dh), row_weights(positions, weights), host(codes).astype(np.float64)
    x = np.concatenate([q[:, :I] * host(scale)[:, :1], q[:, I:] * host(scale)[:, 1:]], 1)

    def loss(x, w):
        g, u = x[:, :I], x[:, I:]
        return (d * w * g * sigmoid64(g) * u).sum()
    e = 1e-6
    for r in range(T * k):
        for c in (0, 7, 39, 40, 63, 79):
            up, down = x.copy(), x.copy()
            up[r, c] += e
            down[r, c] -= e
            num = (loss(up, wr) - loss(down, wr)) / (2 * e)
            assert abs(num - dGU[r, c]) <= 2.0 ** -8 * abs(num) + 1e-7
    at = host(positions)
    for t in range(T):
        for j in range(k):
            up, down = wr.copy(), wr.copy()
            up[at[t, j]] += e
            down[at[t, j]] -= e
            num = (loss(x, up) - loss(x, down)) / (2 * e)
            assert abs(num - dw[t, j]) <= 1e-5 * max(1, abs(num))


def test_rows_that_hold_anything(drgg):
    """A row of weight 0 gives zeros, one with an infinity or NaN has a NaN scale, a position outside the rows is
    skipped and its row left as it was."""
    T, k, I = 4, 2, 144
    GU, positions, weights, dh = make(T, k, I, "normal", 3)
    weights = weights + 0.5
    at = host(positions)
    weights[1, 0] = 0
    GU[at[1, 0]] = float("nan")
    dh[at[1, 0]] = float("inf")
    GU[at[2, 1], 3] = float("inf")
    skipped = int(at[3, 0])
    positions[3, 0] = T * k
    h, codes, scale = drgg.moe_gate_int8(GU, positions, weights)
    assert not host(h)[at[1, 0]].any()
    s = host(scale)
    assert np.isnan(s[at[1, 0]]).all() and np.isnan(s[at[2, 1]]).tolist() == [True, False, False, False]
    assert not host(codes)[at[2, 1], :128].any()
    filled = [torch.full_like(GU, 5), torch.full_like(h, 5), torch.full_like(weights, 5)]
    st = drgg.lib.moe_gate_int8_grad(dh.data_ptr(), codes.data_ptr(), scale.data_ptr(), positions.data_ptr(), weights.data_ptr(),
                                     T, k, I, *(t.data_ptr() for t in filled), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    dGU, h2, dw = (host(t) for t in filled)
    assert not dGU[at[1, 0]].any() and not h2[at[1, 0]].any()
    assert (dGU[skipped] == 5).all() and (h2[skipped] == 5).all() and dw[3, 0] == 0
    others = [p for p in range(T * k) if p not in (skipped, at[1, 0], at[2, 1])]
    assert np.isfinite(dGU[others]).all()


# ---- the training block ---------------------------------------------------------------

def block(T, E, H, I, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, by=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * by).to(dtype).requires_grad_()
    return normal(T, H), normal(T, E, dtype=torch.float32), normal(E, 2 * I, H, by=H ** -0.5), normal(E, H, I, by=I ** -0.5)


@pytest.mark.parametrize("scored", [False, True])
def test_training_block_is_its_parts(drgg, scored):
    from dense_ragged_grouped_amd import moe
    T, E, k, H, I = 130, 6, 3, 72, 136
    X, logits, W1, W2 = block(T, E, H, I)
    bias = torch.linspace(-0.1, 0.1, E, device="cuda")
    sc = drgg.Scoring(bias=bias, groups=3, top_groups=2) if scored else None
    out = moe.ffn(X, logits, W1, W2, k, scoring=sc, kept="int8")
    dout = torch.randn_like(out)
    got = torch.autograd.grad(out, (X, logits, W1, W2), dout)
    with torch.no_grad():
        r = drgg.moe_route_scores(logits, k, sc) if scored else drgg.moe_route(logits, k)
        o = r.group_offsets
        Xg = drgg.moe_dispatch(X, r.positions)
        h, q, s = drgg.moe_gate_int8(drgg.grouped_gemm_fwd(Xg, W1, o), r.positions, r.weights)
        assert torch.equal(out, drgg.moe_combine(drgg.grouped_gemm_fwd(h, W2, o), r.positions))
        drows = drgg.moe_dispatch(dout, r.positions)
        dGU, h, dw = drgg.moe_gate_int8_grad(drgg.grouped_gemm_dgrad(drows, W2, o), q, s, r.positions, r.weights)
        dl = (drgg.moe_route_scores_grad(dw, logits, r.experts, r.weights, sc) if scored else
              drgg.moe_route_grad(dw, logits, r.experts, r.weights))
        want = (drgg.moe_combine(drgg.grouped_gemm_dgrad(dGU, W1, o), r.positions), dl, drgg.grouped_gemm_wgrad(Xg, dGU, o),
                drgg.grouped_gemm_wgrad(h, drows, o))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_training_block_against_the_formula(drgg):
    """Of the block without kept, in 64 bits by autograd.  8-bit codes are off by m / 254 each, m the largest of 128
    (about 2.9 standard deviations): 0.7 % of a standard deviation rms, which moves each gradient's norm by about
    that; BF16 roundings of the passed values (2^-8 at most each, five in a row) are the rest: 3 % in all."""
    from dense_ragged_grouped_amd import moe
    T, E, k, H, I = 200, 4, 2, 128, 256
    X, logits, W1, W2 = block(T, E, H, I, 1)
    out = moe.ffn(X, logits, W1, W2, k, kept="int8")
    dout = torch.randn_like(out)
    got = torch.autograd.grad(out, (X, logits, W1, W2), dout)
    x, l, w1, w2 = (t.detach().double().cpu().requires_grad_() for t in (X, logits, W1, W2))
    top, experts = torch.topk(l, k, dim=1)
    y = 0
    for j in range(k):
        a = torch.stack([w1[e] @ v for e, v in zip(experts[:, j], x)])
        h = torch.nn.functional.silu(a[:, :I]) * a[:, I:]
        y = y + torch.softmax(top, 1)[:, j, None] * torch.stack([w2[e] @ v for e, v in zip(experts[:, j], h)])
    want = torch.autograd.grad(y, (x, l, w1, w2), dout.double().cpu())
    assert float((out.detach().double().cpu() - y.detach()).norm() / y.detach().norm()) < 0.02
    for a, b in zip(got, want):
        assert float((a.double().cpu() - b).norm() / b.norm()) < 0.03


def test_what_the_block_keeps(drgg):
    """Of the experts' rows, the codes and scales alone."""
    from dense_ragged_grouped_amd import moe
    T, E, k, H, I = 256, 4, 2, 128, 256
    X, logits, W1, W2 = block(T, E, H, I)
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        moe.ffn(X, logits, W1, W2, k, kept="int8")
    rows = [(t.dtype, t.shape[1]) for t in kept if t.dim() == 2 and t.shape[0] == T * k]
    assert len(rows) == 2 and set(rows) == {(torch.int8, 2 * I), (torch.float32, 2 * 2)}


def test_only_some_gradients(drgg):
    from dense_ragged_grouped_amd import moe
    X, logits, W1, W2 = block(40, 4, 64, 64)
    full = torch.autograd.grad(moe.ffn(X, logits, W1, W2, 2, kept="int8").float().sum(), (X, logits, W1, W2))
    for i, t in enumerate((X, logits, W1, W2)):
        parts = [u if u is t else u.detach() for u in (X, logits, W1, W2)]
        for graph in (False, True):
            one, = torch.autograd.grad(moe.ffn(*parts, 2, kept="int8").float().sum(), t, create_graph=graph)
            assert torch.equal(one, full[i])


def test_blocks_without_tokens(drgg):
    """No tokens: empty results and zero gradients of the weights, from every block that selects by scores."""
    from dense_ragged_grouped_amd import moe
    E, H, I, k = 4, 64, 32, 2
    sc = drgg.Scoring(bias=torch.zeros(E, device="cuda"), groups=2, top_groups=1)
    X = torch.zeros(0, H, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    logits = torch.zeros(0, E, device="cuda", requires_grad=True)
    W1 = torch.ones(E, 2 * I, H, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    W2 = torch.ones(E, H, I, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    for kept in ("int8", None):
        out = moe.ffn(X, logits, W1, W2, k, scoring=sc, kept=kept)
        assert out.shape == (0, H)
        grads = torch.autograd.grad(out.float().sum(), (X, logits, W1, W2))
        assert [g.shape for g in grads] == [x.shape for x in (X, logits, W1, W2)]
        assert not grads[2].any() and not grads[3].any()
    w1, w2 = W1.detach(), W2.detach()
    for scoring in (sc, None):
        assert moe.ffn_int8(X.detach(), logits.detach(), *moe.quantize_weights(w1), *moe.quantize_weights(w2), k,
                            scoring=scoring).shape == (0, H)
        assert moe.ffn_mxfp4(X.detach(), logits.detach(), *moe.quantize_weights_mxfp4(w1), *moe.quantize_weights_mxfp4(w2), k,
                             scoring=scoring).shape == (0, H)


def test_second_derivative_raises(drgg):
    from dense_ragged_grouped_amd import moe
    X, logits, W1, W2 = block(10, 4, 64, 64)
    g, = torch.autograd.grad(moe.ffn(X, logits, W1, W2, 2, kept="int8").float().pow(2).sum(), W1, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.float().sum().backward()


def test_step_captured_and_replayed(drgg):
    """Forward and backward in a graph, replayed on changing inputs beside eager steps."""
    from dense_ragged_grouped_amd import moe
    X, logits, W1, W2 = (t.detach() for t in block(100, 4, 64, 96))
    dout = torch.randn(100, 64, device="cuda").bfloat16()

    def step():
        leaves = [t.detach().requires_grad_() for t in (X, logits, W1, W2)]
        out = moe.ffn(*leaves, 2, kept="int8")
        return (out.detach(), *torch.autograd.grad(out, leaves, dout))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in (X, logits):
            t.copy_(torch.randn_like(t))
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_on_another_stream(drgg):
    GU, positions, weights, dh = make(20, 2, 264, "normal", 9)
    want = drgg.moe_gate_int8(GU, positions, weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = drgg.moe_gate_int8(GU, positions, weights, stream=side)
    grads = drgg.moe_gate_int8_grad(dh, got[1], got[2], positions, weights, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((*want, *drgg.moe_gate_int8_grad(dh, want[1], want[2], positions, weights)), (*got, *grads)):
        assert torch.equal(a, b)


def test_refusals(drgg):
    from dense_ragged_grouped_amd import moe
    GU, positions, weights, dh = make(4, 2, 24, "normal", 0)
    _, q, s = drgg.moe_gate_int8(GU, positions, weights)
    for bad in (lambda: drgg.moe_gate_int8(GU.float(), positions, weights),
                lambda: drgg.moe_gate_int8(GU[:, :46].contiguous(), positions, weights),
                lambda: drgg.moe_gate_int8(GU[:, :40].contiguous(), positions, weights),   # I = 20
                lambda: drgg.moe_gate_int8(GU[:6], positions, weights),
                lambda: drgg.moe_gate_int8(GU, positions.long(), weights),
                lambda: drgg.moe_gate_int8(GU, positions, weights[:, :1].contiguous()),
                lambda: drgg.moe_gate_int8(GU.t().contiguous().t(), positions, weights),
                lambda: drgg.moe_gate_int8_grad(dh, q[:, :24].contiguous(), s, positions, weights),
                lambda: drgg.moe_gate_int8_grad(dh, q, s[:, :1].contiguous(), positions, weights),
                lambda: drgg.moe_gate_int8_grad(dh, q.to(torch.uint8), s, positions, weights),
                lambda: moe.ffn(*block(4, 4, 64, 64), 2, kept="fp8")):
        with pytest.raises((TypeError, ValueError, drgg.DrggError)):
            bad()


def test_every_quotient(drgg):
    """Codes of every BF16 value from 2^-9 to 1 times a block's largest, for every significand of that, at scales from
    FP32's smallest to its largest: those of the exact quotient, ties to even."""
    x = (np.arange(128, 256)[None, :] * np.exp2(-7.0 - np.arange(10))[:, None]).reshape(-1)   # [2^-9, 2)
    for shift in (-126.0, -70.0, 0.0, 99.0, 126.0):
        rows = []
        for m in np.arange(128, 256) / 128:
            v = x[x <= m]
            v = np.concatenate([v, np.zeros(-len(v) % 127)]).reshape(-1, 127)
            rows.append(np.concatenate([np.full((len(v), 1), m), v * np.where(np.arange(127) % 2, -1, 1)], 1))
        g = np.concatenate(rows) * 2.0 ** shift
        g = np.where(np.abs(g) < 2.0 ** -133, 0, g).astype(np.float32)
        GU = dev(np.concatenate([g, g[:, ::-1]], 1)).bfloat16()
        R = len(g)
        positions, weights = torch.arange(R, dtype=torch.int32, device="cuda").view(R, 1), torch.ones(R, 1, device="cuda")
        _, codes, scale = drgg.moe_gate_int8(GU, positions, weights)
        gu = host(GU)
        want = [kept64(gu[:, :128]), kept64(gu[:, 128:])]
        assert np.array_equal(host(codes), np.concatenate([w[0] for w in want], 1))
        assert np.array_equal(scale.cpu().numpy(), np.concatenate([w[1] for w in want], 1))
