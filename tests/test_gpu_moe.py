"""The router's selection, the movement of rows and the training block on the
GPU, against plain implementations in 64 bits (NumPy).

Tolerances.  u = 2^-24 (FP32), each derived from the operator's steps:
* softmax weights: the argument l - max is rounded once (relative u, so the
  term moves by |l - max| u), exp is within 2 ulp, and the sum of n positive
  terms in a tree within log2(n) u: relative error at most
  (|l - max| + 2 log2(n) + 8) u, doubled for the second-order terms.
* their gradient: products and sums of k (or E) such values: the same
  relative error on every factor, so 8 of them bound the sum of magnitudes.
* combine: k products and sums, (k + 1) u of the sum of magnitudes, and one
  rounding (half the spacing of the type at the value).
* combine's dweights: at most H roundings in any order, H u of the sum of
  magnitudes; drows: one product and one rounding.
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


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def spacing(v, dtype):
    """Half the distance between neighbouring values of the type at v: 8
    significant bits (BF16) or 24 (FP32)."""
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    return half * np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))))


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


# ---- selection -----------------------------------------------------------------

def choose(logits, k):
    """(experts, positions, offsets) by Python's own sorts: value decreasing
    (NaN first), index increasing; pairs stably by expert."""
    T, E = logits.shape
    nan = np.isnan(logits)
    value = np.where(nan, 0.0, logits) + 0.0
    experts = np.empty((T, k), dtype=np.int64)
    for t in range(T):
        experts[t] = sorted(range(E), key=lambda e: (not nan[t, e], -value[t, e], e))[:k]
    flat = experts.reshape(-1)
    order = sorted(range(T * k), key=lambda p: (flat[p], p))
    positions = np.empty(T * k, dtype=np.int64)
    positions[order] = np.arange(T * k)
    offsets = np.searchsorted(flat[order], np.arange(E + 1)) if T else np.zeros(E + 1)
    return experts, positions.reshape(T, k), offsets


def softmax64(v):
    """Rows of -inf alone give zeros."""
    with np.errstate(invalid="ignore"):
        most = v.max(1, keepdims=True) if v.size else v[:, :1]
        p = np.exp(v - np.where(np.isneginf(most), 0.0, most))
        total = p.sum(1, keepdims=True)
        return np.where(total == 0, 0.0, p / np.where(total == 0, 1.0, total))


def weights64(logits, experts, renormalize):
    l64 = logits.astype(np.float64)
    chosen = np.take_along_axis(l64, experts, 1)
    return softmax64(chosen) if renormalize else np.take_along_axis(softmax64(l64), experts, 1)


def weight_tolerance(logits, experts):
    with np.errstate(invalid="ignore"):
        chosen = np.take_along_axis(logits.astype(np.float64), experts, 1)
        far = np.abs(chosen - chosen[:, :1])
    far = np.where(np.isfinite(far), far, 0.0)
    return 2 * (far + 2 * np.log2(logits.shape[1] + 1) + 8) * U


def make_logits(kind, T, E, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, E)).astype(np.float32)
    if kind == "ties":
        x = rng.integers(-2, 3, (T, E)).astype(np.float32)
        x[x == 0] *= np.where(rng.random((x == 0).sum()) < 0.5, -1, 1)   # both zeros
    elif kind == "masked":
        x[rng.random((T, E)) < 0.8] = -np.inf
        x[::3] = -np.inf
    elif kind == "lowest":
        x[rng.random((T, E)) < 0.8] = np.finfo(np.float32).min
        x[::3] = np.finfo(np.float32).min
    elif kind == "wide":
        x *= 30
    elif kind == "tiny":
        x *= np.float32(1e-40)
    return x


SHAPES = [(0, 8, 2), (1, 1, 1), (1, 256, 8), (2, 3, 3), (63, 8, 2), (64, 100, 5), (65, 32, 4), (130, 257, 8),
          (193, 511, 7), (515, 1024, 64), (1030, 1000, 6), (4099, 64, 8)]


@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "lowest", "wide", "tiny"])
@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(drgg, T, E, k, kind, renormalize):
    logits = make_logits(kind, T, E, 7 * T + E + k)
    r = drgg.moe_route(dev(logits), k, renormalize=renormalize)
    experts, positions, offsets = choose(logits, k)
    assert np.array_equal(host(r.experts), experts)
    assert np.array_equal(host(r.positions), positions)
    assert np.array_equal(host(r.group_offsets), offsets)
    assert np.array_equal(host(r.tokens)[positions.reshape(-1)], np.repeat(np.arange(T), k))
    w, want = host(r.weights), weights64(logits, experts, renormalize)
    assert np.all(np.abs(w - want) <= weight_tolerance(logits, experts) * want + 2.0 ** -126)
    if kind == "masked":
        assert not w[np.isneginf(np.take_along_axis(logits, experts, 1))].any()


@pytest.mark.parametrize("kind", ["normal", "ties"])
@pytest.mark.parametrize("T,E,k", [(32768, 7, 3), (32769, 130, 2), (70001, 6, 1)])
def test_route_many_tokens(drgg, T, E, k, kind):
    logits = make_logits(kind, T, E, T + E)
    r = drgg.moe_route(dev(logits), k)
    experts = np.argsort(-(logits + 0.0), axis=1, kind="stable")[:, :k]
    flat = experts.reshape(-1)
    order = np.argsort(flat, kind="stable")
    positions = np.empty(T * k, dtype=np.int64)
    positions[order] = np.arange(T * k)
    assert np.array_equal(host(r.experts), experts)
    assert np.array_equal(host(r.positions).reshape(-1), positions)
    assert np.array_equal(host(r.tokens), order // k)
    assert np.array_equal(host(r.group_offsets), np.searchsorted(flat[order], np.arange(E + 1)))


def test_route_nan_and_infinity(drgg):
    """NaN sorts first (either sign), then +inf; their softmax is NaN, and no other token's is."""
    logits = make_logits("normal", 70, 40, 3)
    logits[5, 7] = np.nan
    logits[9, 39] = np.uint32(0xFFC00001).view(np.float32)
    logits[11, [3, 20]] = np.inf
    for renormalize in (True, False):
        r = drgg.moe_route(dev(logits), 4, renormalize=renormalize)
        experts, positions, offsets = choose(logits, 4)
        assert np.array_equal(host(r.experts), experts) and np.array_equal(host(r.positions), positions)
        assert experts[5, 0] == 7 and experts[9, 0] == 39 and list(experts[11, :2]) == [3, 20]
        w = host(r.weights)
        assert np.isnan(w[[5, 9]]).all() and np.isnan(w[11, :2]).all()
        others = [t for t in range(70) if t not in (5, 9, 11)]
        assert np.isfinite(w[others]).all()


def test_route_is_a_pure_function(drgg):
    """Same bits on repeated calls, on another stream, with a caller's workspace full of garbage, and under graph replay."""
    logits = dev(make_logits("ties", 3001, 128, 5))
    first = drgg.moe_route(logits, 6)
    nbytes = drgg.route_workspace_size(3001, 128, 6)
    assert nbytes > 0 and drgg.route_workspace_size(64, 128, 6) == 0
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [drgg.moe_route(logits, 6), drgg.moe_route(logits, 6, workspace=ws), drgg.moe_route(logits, 6, stream=side)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = drgg.moe_route(logits, 6, workspace=ws)
    for _ in range(3):
        for t in captured:
            t.zero_()
        drgg.moe_route(logits, 5)
        g.replay()
        torch.cuda.synchronize()
        again.append([t.clone() for t in captured])
    for other in again:
        for a, b in zip(first, other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["normal", "masked", "wide"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 5, 5), (67, 100, 4), (130, 512, 8), (9, 1023, 64)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_grad_against_the_formula(drgg, T, E, k, kind, renormalize):
    logits = make_logits(kind, T, E, T + E + k)
    dw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    r = drgg.moe_route(dev(logits), k, renormalize=renormalize)
    got = host(drgg.moe_route_grad(dev(dw), dev(logits), r.experts, r.weights, renormalize=renormalize))
    experts, d = choose(logits, k)[0], dw.astype(np.float64)
    w = weights64(logits, experts, renormalize)
    inner = (w * d).sum(1, keepdims=True)
    size = (w * np.abs(d)).sum(1, keepdims=True)
    if renormalize:
        want, mag = np.zeros((T, E)), np.zeros((T, E))
        np.put_along_axis(want, experts, w * (d - inner), 1)
        np.put_along_axis(mag, experts, w * (np.abs(d) + size), 1)
    else:
        p, at = softmax64(logits.astype(np.float64)), np.zeros((T, E))
        np.put_along_axis(at, experts, d, 1)
        want, mag = p * (at - inner), p * (np.abs(at) + size)
    far = np.where(np.isfinite(logits), logits, 0).astype(np.float64)
    tol = 8 * 2 * (np.ptp(far, axis=1, keepdims=True) + 2 * np.log2(E + 1) + 8 + k) * U
    assert np.all(np.abs(got - want) <= tol * mag + 2.0 ** -120)
    if kind == "masked":
        assert not got[np.isneginf(logits)].any()


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_grad_against_differences(drgg, renormalize):
    """Central differences of sum(dw * weights) with a step of 2^-6 on logits
    whose order it cannot change: truncation at most step^2/6 times a third
    derivative below 6 sum|dw|, rounding 2u sum|dw| / step."""
    T, E, k, step = 4, 12, 4, 2.0 ** -6
    rng = np.random.default_rng(2)
    logits = np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float32) * 0.25
    dw = rng.standard_normal((T, k)).astype(np.float32)
    r = drgg.moe_route(dev(logits), k, renormalize=renormalize)
    got = host(drgg.moe_route_grad(dev(dw), dev(logits), r.experts, r.weights, renormalize=renormalize))
    size = np.abs(dw).sum(1)
    for e in range(E):
        f = []
        for sign in (1, -1):
            moved = logits.copy()
            moved[:, e] += sign * step
            f.append((host(drgg.moe_route(dev(moved), k, renormalize=renormalize).weights) * dw).sum(1))
        diff = (f[0] - f[1]) / (2 * step)
        assert np.all(np.abs(got[:, e] - diff) <= size * (step ** 2 + 40 * U / step))


# ---- rows ------------------------------------------------------------------------

def permutation(T, k, seed):
    return np.random.default_rng(seed).permutation(T * k).reshape(T, k).astype(np.int32)


def row_values(shape, dtype, seed):
    t = dev(np.random.default_rng(seed).standard_normal(shape).astype(np.float32), dtype)
    return t, host(t)


ROWS = [(0, 2, 64), (1, 1, 8), (1, 8, 2048), (3, 64, 40), (5, 3, 776), (17, 8, 4104), (33, 2, 128), (257, 6, 264)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H", ROWS)
def test_dispatch_and_combine(drgg, T, k, H, dtype):
    positions = permutation(T, k, T + k)
    X, x = row_values((T, H), dtype, 1)
    rows = drgg.moe_dispatch(X, dev(positions))
    want = np.empty((T * k, H))
    want[positions.reshape(-1)] = np.repeat(x, k, 0)
    assert np.array_equal(host(rows), want)
    R, r = row_values((T * k, H), dtype, 2)
    w = np.random.default_rng(3).standard_normal((T, k)).astype(np.float32)
    for weights in (None, w):
        got = host(drgg.moe_combine(R, dev(positions), None if weights is None else dev(weights)))
        terms = r[positions] * (1.0 if weights is None else weights.astype(np.float64)[:, :, None])
        want, size = terms.sum(1), np.abs(terms).sum(1)
        before = (k + 1) * U * size
        assert np.all(np.abs(got - want) <= before + spacing(np.abs(want) + before, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H", ROWS)
def test_combine_grad(drgg, T, k, H, dtype):
    positions = permutation(T, k, 5 * T + k)
    R, r = row_values((T * k, H), dtype, 4)
    G, g = row_values((T, H), dtype, 5)
    w = np.random.default_rng(6).standard_normal((T, k)).astype(np.float32)
    drows, dweights = drgg.moe_combine_grad(G, R, dev(positions), dev(w))
    want = np.empty((T * k, H))
    want[positions.reshape(-1)] = (w.astype(np.float64)[:, :, None] * g[:, None, :]).reshape(T * k, H)
    assert np.all(np.abs(host(drows) - want) <= 2 * U * np.abs(want) + spacing((1 + 2 * U) * want, dtype))
    terms = r[positions] * g[:, None, :]
    assert np.all(np.abs(host(dweights) - terms.sum(2)) <= H * U * np.abs(terms).sum(2))
    again = drgg.moe_combine_grad(G, R, dev(positions), dev(w))
    assert torch.equal(drows, again[0]) and torch.equal(dweights, again[1])


def test_many_tokens_and_long_buffers(drgg):
    """Rows beyond 2^31 values and 2^32 bytes, and more tokens than a launch has blocks: with weights 1/4 the sum of
    four copies of a row is the row."""
    T, k, H = 140001, 4, 4096
    X = torch.randn((T, H), device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    positions = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    rows = drgg.moe_dispatch(X, positions)
    assert torch.equal(rows[positions[-1].long()], X[-1:].expand(k, H))
    w = torch.full((T, k), 0.25, device="cuda")
    assert torch.equal(drgg.moe_combine(rows, positions, w), X)
    drows, dweights = drgg.moe_combine_grad(X, rows, positions, w)
    assert torch.equal(drows[positions[:, 3].long()], X * 0.25)
    few = [0, 70000, T - 1]
    want = X[few].double().square().sum(1, keepdim=True).expand(-1, k)
    assert torch.all((dweights[few].double() - want).abs() <= H * U * want)


def test_long_logits(drgg):
    """Logits beyond 2^31 values: the last tokens are chosen as in a small call."""
    T, E, k = 2200000, 1024, 2
    logits = torch.randn((T, E), device="cuda")
    r = drgg.moe_route(logits, k)
    last = drgg.moe_route(logits[-50:], k)
    assert torch.equal(r.experts[-50:], last.experts) and torch.equal(r.weights[-50:], last.weights)
    counts = torch.bincount(r.experts.flatten(), minlength=E)
    assert torch.equal(r.group_offsets[1:].long(), counts.cumsum(0)) and int(r.group_offsets[0]) == 0
    at = r.positions.flatten().long()
    assert torch.equal(torch.bincount(at, minlength=T * k), torch.ones_like(at))
    assert torch.equal(r.tokens[at], torch.arange(T, device="cuda", dtype=torch.int32).repeat_interleave(k))
    by_row = torch.empty_like(at)
    by_row[at] = r.experts.flatten().long()
    assert bool((by_row[1:] >= by_row[:-1]).all())
    same = by_row[1:] == by_row[:-1]
    assert bool((r.tokens[1:] > r.tokens[:-1])[same].all())
    d = drgg.moe_route_grad(torch.ones_like(r.weights), logits, r.experts, r.weights)
    assert float(d[-50:].abs().max()) <= 8 * U


def test_masked_pairs_do_not_spread_nan(drgg):
    """An entry outside the rows is skipped: its row's NaN does not reach the sum, and nothing is written through it."""
    T, k, H = 6, 3, 48
    positions = permutation(T, k, 1)
    R, r = row_values((T * k, H), torch.float32, 2)
    R[int(positions[2, 1])] = float("nan")
    skip = positions.copy()
    skip[2, 1], skip[4, 0] = -1, T * k
    w = dev(np.ones((T, k), dtype=np.float32))
    got = host(drgg.moe_combine(R, dev(skip), w))
    assert np.isfinite(got).all()
    out = torch.full((T * k, H), 7.0, device="cuda")
    drgg.moe_dispatch(torch.zeros((T, H), device="cuda"), dev(skip), out=out)
    left = np.setdiff1d(np.arange(T * k), skip.reshape(-1))
    out = host(out)
    assert len(left) == 2 and (out[left] == 7.0).all() and not np.delete(out, left, 0).any()
    _, dweights = drgg.moe_combine_grad(torch.ones((T, H), device="cuda"), R, dev(skip), w)
    assert host(dweights)[2, 1] == 0 and host(dweights)[4, 0] == 0 and np.isfinite(host(dweights)).all()


def test_combine_grad_against_differences(drgg):
    """The sum is linear in rows and weights: differences in FP32 are exact up to rounding (values and steps of a few bits)."""
    T, k, H = 5, 3, 24
    rng = np.random.default_rng(8)
    positions = permutation(T, k, 8)
    r, w, g = (rng.integers(-8, 9, s).astype(np.float32) / 8 for s in ((T * k, H), (T, k), (T, H)))
    drows, dweights = (host(t) for t in drgg.moe_combine_grad(dev(g), dev(r), dev(positions), dev(w)))

    def f(rows, weights):
        return (host(drgg.moe_combine(dev(rows), dev(positions), dev(weights))) * g).sum()
    for t, j in ((0, 0), (2, 1), (4, 2)):
        up = w.copy()
        up[t, j] += 1
        assert f(r, up) - f(r, w) == dweights[t, j]
    for i, h in ((0, 0), (7, 11), (14, 23)):
        up = r.copy()
        up[i, h] += 1
        assert f(up, w) - f(r, w) == drows[i, h]


# ---- the training block -----------------------------------------------------------

def test_ffn_trains(drgg):
    """Outputs and all four gradients of the BF16 block against 64 bits.  The
    hidden rows and the experts' outputs are rounded to BF16 between the
    operators (three roundings forward, about as many back, each at most 2^-8 of
    a value): 2 % of the result's norm bounds them with room."""
    from dense_ragged_grouped_amd import moe
    T, E, k, H, I = 150, 6, 2, 64, 48
    rng = np.random.default_rng(12)
    X = dev(rng.standard_normal((T, H)).astype(np.float32), torch.bfloat16).requires_grad_(True)
    logits = dev(rng.standard_normal((T, E)).astype(np.float32)).requires_grad_(True)
    W1 = dev((rng.standard_normal((E, 2 * I, H)) / 8).astype(np.float32), torch.bfloat16).requires_grad_(True)
    W2 = dev((rng.standard_normal((E, H, I)) / 7).astype(np.float32), torch.bfloat16).requires_grad_(True)
    G = dev(rng.standard_normal((T, H)).astype(np.float32), torch.bfloat16)
    out = moe.ffn(X, logits, W1, W2, k)
    grads = torch.autograd.grad(out, (X, logits, W1, W2), G)
    leaves = [t.detach().double().cpu().requires_grad_(True) for t in (X, logits, W1, W2)]
    x, l, w1, w2 = leaves
    top, experts = torch.topk(l, k, dim=1)
    w = torch.softmax(top, 1)
    want = 0
    for j in range(k):
        h = torch.einsum("th,tnh->tn", x, w1[experts[:, j]])
        h = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        want = want + w[:, j, None] * torch.einsum("ti,thi->th", h, w2[experts[:, j]])
    for got, ref in zip((out, *grads), (want, *torch.autograd.grad(want, leaves, G.double().cpu()))):
        err = (got.detach().double().cpu() - ref).norm() / ref.norm()
        assert err < 0.02, float(err)


# ---- refusals -----------------------------------------------------------------------

def test_refusals(drgg):
    logits = torch.zeros((4, 8), device="cuda")
    for bad in (0, 9, 65):
        with pytest.raises(drgg.DrggError):
            drgg.moe_route(logits, bad)
    with pytest.raises(drgg.DrggError):
        drgg.moe_route(torch.zeros((4, 1025), device="cuda"), 2)
    with pytest.raises(TypeError):
        drgg.moe_route(logits.bfloat16(), 2)
    with pytest.raises(TypeError):
        drgg.moe_route(logits.cpu(), 2)
    with pytest.raises(ValueError):
        drgg.moe_route(torch.zeros((8, 4), device="cuda").t(), 2)
    with pytest.raises(drgg.DrggError):   # not 16-byte aligned
        drgg.moe_route(torch.zeros(4 * 8 + 1, device="cuda")[1:].view(4, 8), 2)
    big = torch.zeros((130, 8), device="cuda")
    with pytest.raises(drgg.DrggError):   # workspace missing
        drgg.moe_route(big, 2, workspace=False)
    r = drgg.moe_route(logits, 2)
    with pytest.raises(ValueError):
        drgg.moe_route_grad(r.weights[:2].contiguous(), logits, r.experts, r.weights)
    X = torch.zeros((4, 24), device="cuda")
    with pytest.raises(TypeError):
        drgg.moe_dispatch(X.half(), r.positions)
    with pytest.raises(drgg.DrggError):
        drgg.moe_dispatch(torch.zeros((4, 20), device="cuda"), r.positions)
    with pytest.raises(ValueError):
        drgg.moe_dispatch(X[:3], r.positions)
    with pytest.raises(TypeError):
        drgg.moe_dispatch(X, r.positions.long())
    rows = drgg.moe_dispatch(X, r.positions)
    with pytest.raises(ValueError):
        drgg.moe_combine(rows[:6], r.positions)
    with pytest.raises(ValueError):
        drgg.moe_combine(rows, r.positions, r.weights, out=torch.empty((4, 16), device="cuda"))
    with pytest.raises(ValueError):
        drgg.moe_combine_grad(rows, rows, r.positions, r.weights)
    with pytest.raises(ValueError):
        drgg.moe_combine(rows, r.positions, r.weights.t().contiguous().t())
