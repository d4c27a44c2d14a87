"""The 8-bit integer products on the GPU, against exact integer products
scaled in 64 bits.

Tolerances.  u = 2^-24: the sum is exact; turning it into FP32 and the two
scales are three roundings, 3 u of the value (4 u with second-order terms),
and the output's rounding half the spacing of its type at the value.  The gate adds exp within 2 ulp,
a sum, a division and a product, and g itself enters exp with an error of
|g| 4 u: (4 |g| + 16) u of the value.  Codes are compared with the same IEEE
FP32 operations in NumPy, exactly, and with 64 bits to half a step plus the
roundings of 127 x / max (256 u of a step).
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


# ---- quantisation ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K", [(0, 64), (1, 16), (1, 4096), (3, 48), (7, 2064), (130, 768), (5, 20000)])
def test_quantize(drgg, T, K, dtype):
    rng = np.random.default_rng(T + K)
    X = dev(rng.standard_normal((T, K)).astype(np.float32) * np.exp2(rng.integers(-30, 30, (T, 1))).astype(np.float32),
            dtype)
    if T > 2:
        X[1] = 0
        X[2, ::2] = -X[2].abs().max() / 2      # ties at 63.5
    q, s = drgg.quantize_int8(X)
    x = X.float().cpu().numpy()
    most = np.abs(x).max(1, keepdims=True) if T else np.zeros((0, 1), np.float32)
    by = np.where(most == 0, np.float32(1), most)
    assert np.array_equal(host(q), np.rint(x * np.float32(127) / by))
    assert np.array_equal(s.cpu().numpy(), (most / np.float32(127))[:, 0])
    exact = 127 * x.astype(np.float64) / by
    assert np.all(np.abs(host(q) - exact) <= 0.5 + 127 * 2 * U)
    if T > 2:
        assert not host(q)[1].any() and host(s)[1] == 0


def test_quantize_extremes(drgg):
    """Infinity and NaN mark their own row; the largest and smallest values keep their codes."""
    X = np.random.default_rng(1).standard_normal((8, 64)).astype(np.float32)
    X[1, 5], X[2, 6], X[3, 7] = np.inf, -np.inf, np.nan
    X[4] *= np.float32(2.0 ** 125)
    X[5] = 0
    X[5, 3], X[5, 4] = np.float32(2.0 ** -149), np.float32(2.0 ** -149) * 2
    q, s = (host(t) for t in drgg.quantize_int8(dev(X)))
    assert np.isnan(s[1:4]).all() and not q[1:4].any()
    assert np.isfinite(s[[0, 4, 5, 6, 7]]).all()
    assert np.all(np.abs(q[4] - 127 * X[4].astype(np.float64) / np.abs(X[4]).max()) <= 0.5 + 127 * 2 * U)
    assert list(q[5, 2:6]) == [0, 64, 127, 0]
    y = drgg.gemm_int8(dev(q.astype(np.int8)), dev(s.astype(np.float32)), torch.ones((8, 64), dtype=torch.int8, device="cuda"),
                       torch.ones(8, device="cuda"), out_dtype=torch.float32)
    y = host(y)
    assert np.isnan(y[1:4]).all() and np.isfinite(y[[0, 4, 5, 6, 7]]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,K", [(1, 8, 2048), (9, 3, 80), (40, 2, 1040)])
def test_quantize_into_the_grouped_order(drgg, T, k, K, dtype):
    rng = np.random.default_rng(T)
    X = dev(rng.standard_normal((T, K)).astype(np.float32), dtype)
    positions = rng.permutation(T * k).reshape(T, k).astype(np.int32)
    q0, s0 = drgg.quantize_int8(X)
    q, s = drgg.quantize_int8(X, dev(positions))
    at = torch.from_numpy(positions.reshape(-1)).long().cuda()
    assert torch.equal(q[at], q0.repeat_interleave(k, 0)) and torch.equal(s[at], s0.repeat_interleave(k, 0))


# ---- products ------------------------------------------------------------------------

def operands(M, N, K, E, seed, full=False):
    rng = np.random.default_rng(seed)
    if full:   # the largest magnitudes: every product 2^14
        X, W = np.full((M, K), -128, np.int8), np.full((E, N, K), -128, np.int8)
    else:
        X = rng.integers(-128, 128, (M, K)).astype(np.int8)
        W = rng.integers(-128, 128, (E, N, K)).astype(np.int8)
    xs = rng.uniform(0.5, 2, M).astype(np.float32) / 64
    ws = rng.uniform(0.5, 2, (E, N)).astype(np.float32) / 64
    return X, xs, W, ws


def product64(X, xs, W, ws):
    """Float64 holds the integer sums exactly (below 2^53)."""
    return (X.astype(np.float64) @ W.astype(np.float64).T) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)


def grouped64(X, xs, W, ws, offsets):
    out = np.zeros((len(X), W.shape[1]))
    for e in range(len(W)):
        lo, hi = offsets[e], offsets[e + 1]
        out[lo:hi] = product64(X[lo:hi], xs[lo:hi], W[e], ws[e])
    return out


def check(got, want, dtype, gated):
    if gated:
        I = want.shape[1] // 2
        g, u = want[:, :I], want[:, I:]
        want = g / (1 + np.exp(-g)) * u
        tol = (4 * np.abs(g) + 16) * U
        # below -88 the sigmoid leaves FP32's range: the result is under 2^-100 |g u|
        floor = np.where(g < -80, np.abs(g * u) * 2.0 ** -100, 0) + 2.0 ** -126
    else:
        tol, floor = 4 * U, 0.0
    assert got.shape == want.shape
    err = np.abs(got - want)
    before = tol * np.abs(want) + floor
    assert np.all(err <= before + spacing(np.abs(want) + before, dtype)), float((err / (np.abs(want) + 1e-30)).max())


COUNTS = [[1], [0, 3, 0, 0, 17, 1], [16, 0, 33, 15], [130, 5, 64], [0, 0], [300, 1, 0, 127, 128, 129], [257] * 3 + [0]]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(16, 16), (48, 80), (272, 208), (528, 1040)])
@pytest.mark.parametrize("counts", COUNTS, ids=[str(i) for i in range(len(COUNTS))])
def test_grouped(drgg, counts, N, K, dtype, gated):
    E, M = len(counts), sum(counts)
    X, xs, W, ws = operands(M, N, K, E, M + N + K)
    if gated:   # gates of a few units
        xs = xs / np.float32(16 * np.sqrt(K))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    got = drgg.grouped_gemm_int8(dev(X), dev(xs), dev(W), dev(ws), dev(offsets), gated=gated, out_dtype=dtype)
    check(host(got), grouped64(X, xs, W, ws, offsets), dtype, gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [0, 1, 2, 15, 16, 17, 33, 64, 65, 129, 300, 520])
@pytest.mark.parametrize("N,K", [(16, 4096), (1040, 144)])
def test_dense(drgg, M, N, K, gated):
    X, xs, W, ws = operands(M, N, K, 1, M + N)
    if gated:
        xs = xs / np.float32(16 * np.sqrt(K))
    got = drgg.gemm_int8(dev(X), dev(xs), dev(W[0]), dev(ws[0]), gated=gated, out_dtype=torch.float32)
    check(host(got), product64(X, xs, W[0], ws[0]), torch.float32, gated)
    one = drgg.grouped_gemm_int8(dev(X), dev(xs), dev(W), dev(ws), dev(np.array([0, M], np.int32)), gated=gated,
                                 out_dtype=torch.float32)
    assert torch.equal(got, one)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tile", [1, 2, 4])
@pytest.mark.parametrize("counts,N,K", [([1], 16, 16), ([0, 130, 5, 64], 48, 80), ([300, 1, 0, 257, 128], 528, 1040),
                                        ([9] * 70, 272, 336), ([2000, 3000], 1040, 272)])
def test_every_tile(drgg, counts, N, K, tile, gated):
    """Each output tile, forced, gives the bits of the program chosen for the sizes (the sums are exact and scaled in one
    way), and the exact product within the tolerance; with and without gathered rows."""
    E, M = len(counts), sum(counts)
    X, xs, W, ws = operands(M, N, K, E, M + K)
    if gated:
        xs = xs / np.float32(16 * np.sqrt(K))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    args = [dev(a) for a in (X, xs, W, ws, offsets)]
    rows = torch.randperm(M, device="cuda").to(torch.int32)
    back = torch.argsort(rows)
    for dtype in (torch.bfloat16, torch.float32):
        free = drgg.grouped_gemm_int8(*args, gated=gated, out_dtype=dtype)
        drgg.set_knob(drgg.KNOB_TILE, tile)
        try:
            got = drgg.grouped_gemm_int8(*args, gated=gated, out_dtype=dtype)
            gathered = drgg.grouped_gemm_int8(args[0][rows.long()], args[1][rows.long()], *args[2:], gated=gated,
                                              rows=back.to(torch.int32), out_dtype=dtype)
        finally:
            drgg.set_knob(drgg.KNOB_TILE, 0)
        assert torch.equal(got, free) and torch.equal(gathered, free)
        check(host(got), grouped64(X, xs, W, ws, offsets), dtype, gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(1040, 208), (2064, 16), (1040, 528)])
def test_many_rows(drgg, N, K, dtype, gated):
    """Enough output tiles that every compute unit has one of the largest."""
    counts = [5000, 0, 1, 7777, 256, 511, 3000]
    M, E = sum(counts), len(counts)
    X, xs, W, ws = operands(M, N, K, E, N + K)
    if gated:
        xs = xs / np.float32(16 * np.sqrt(K))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    out = torch.full((M + 3, N // 2 if gated else N), 7.0, dtype=dtype, device="cuda")
    got = drgg.grouped_gemm_int8(dev(X), dev(xs), dev(W), dev(ws), dev(offsets), gated=gated, out_dtype=dtype, out=out[:M])
    check(host(got), grouped64(X, xs, W, ws, offsets), dtype, gated)
    assert bool((out[M:] == 7.0).all())


@pytest.mark.parametrize("M", [1, 40, 300])
def test_longest_sum_of_the_largest_codes(drgg, M):
    """K = 131056 products of 2^14 stay below 2^31."""
    X, xs, W, ws = operands(M, 16, 131056, 1, M, full=True)
    got = drgg.gemm_int8(dev(X), dev(xs), dev(W[0]), dev(ws[0]), out_dtype=torch.float32)
    check(host(got), product64(X, xs, W[0], ws[0]), torch.float32, False)


@pytest.mark.parametrize("counts", [[3, 0, 9], [200, 0, 300]])
def test_rows_do_not_depend_on_their_company(drgg, counts):
    """A token's result is the same bits alone, in a small group and in a large one; rows past the last group are not written."""
    M, N, K = sum(counts), 144, 336
    X, xs, W, ws = operands(M + 5, N, K, 3, 9)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    out = torch.full((M + 5, N), 7.0, dtype=torch.float32, device="cuda")
    drgg.grouped_gemm_int8(dev(X), dev(xs), dev(W), dev(ws), dev(offsets), out_dtype=torch.float32, out=out)
    assert bool((out[M:] == 7.0).all())
    for t in (0, counts[0] - 1, M - 1):
        e = 0 if t < counts[0] else 2
        alone = drgg.gemm_int8(dev(X[t:t + 1]), dev(xs[t:t + 1]), dev(W[e]), dev(ws[e]), out_dtype=torch.float32)
        assert torch.equal(alone[0], out[t])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,counts,N,K", [(3, [1, 0, 2], 48, 80), (40, [70, 0, 3, 7], 272, 336),
                                          (500, [700, 260, 40], 144, 208), (900, [9000, 1, 7000], 1040, 144)])
def test_gathered_rows(drgg, T, counts, N, K, dtype, gated):
    """rows= gives the same bits as the rows copied out, in every program; an index outside is a row of zeros."""
    rng = np.random.default_rng(T + N)
    M, E = sum(counts), len(counts)
    X, xs, W, ws = (dev(a) for a in operands(T, N, K, E, T + K))
    offsets = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    rows = rng.integers(0, T, M).astype(np.int32)
    at = torch.from_numpy(rows).long().cuda()
    want = drgg.grouped_gemm_int8(X[at], xs[at], W, ws, offsets, gated=gated, out_dtype=dtype)
    got = drgg.grouped_gemm_int8(X, xs, W, ws, offsets, gated=gated, rows=dev(rows), out_dtype=dtype)
    assert torch.equal(got, want)
    bad = rng.choice(M, max(1, M // 50), replace=False)
    rows[bad] = rng.choice([-1, T, 2 ** 31 - 1, -2 ** 31], len(bad))
    got = drgg.grouped_gemm_int8(X, xs, W, ws, offsets, gated=gated, rows=dev(rows), out_dtype=dtype)
    want[torch.from_numpy(bad).cuda()] = 0
    assert torch.equal(got, want)


def test_graph_and_stream(drgg):
    X, xs, W, ws = (dev(a) for a in operands(70, 64, 256, 2, 4))
    offsets = dev(np.array([0, 50, 70], np.int32))
    first = drgg.grouped_gemm_int8(X, xs, W, ws, offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = drgg.grouped_gemm_int8(X, xs, W, ws, offsets, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(first, other)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(first)
    with torch.cuda.graph(g):
        drgg.grouped_gemm_int8(X, xs, W, ws, offsets, out=out)
    for _ in range(3):
        out.zero_()
        drgg.grouped_gemm_int8(X, xs, W, ws, offsets)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)


def test_long_buffers(drgg):
    """Codes and results beyond 2^32 bytes: the last rows as in a small call."""
    M, N, K = 300007, 4096, 16384
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    X = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)
    q, s = drgg.quantize_int8(X)
    few = drgg.quantize_int8(X[-70:].contiguous())
    assert torch.equal(q[-70:], few[0]) and torch.equal(s[-70:], few[1])
    W = torch.randint(-127, 128, (2, N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand((2, N), generator=g, device="cuda")
    offsets = torch.tensor([0, 9, M], dtype=torch.int32, device="cuda")
    y = drgg.grouped_gemm_int8(q, s, W, ws, offsets, out_dtype=torch.float32)
    assert torch.equal(y[-70:], drgg.gemm_int8(q[-70:], s[-70:], W[1], ws[1], out_dtype=torch.float32))
    assert torch.equal(y[:9], drgg.gemm_int8(q[:9], s[:9], W[0], ws[0], out_dtype=torch.float32))


@pytest.mark.parametrize("T,H", [(16500, 131056)])
def test_ffn_too_large_to_gather(drgg, T, H):
    """T * H beyond 2^31: the block copies its tokens into the grouped order
    instead.  Rows do not depend on their company: the first and the last
    tokens give the same bits in a small call."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    X = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn((T, 2), generator=g, device="cuda")
    w1 = torch.randint(-127, 128, (2, 32, H), generator=g, device="cuda", dtype=torch.int8)
    w2 = torch.randint(-127, 128, (2, H, 16), generator=g, device="cuda", dtype=torch.int8)
    s1, s2 = torch.full((2, 32), 1e-4, device="cuda"), torch.full((2, H), 1e-3, device="cuda")
    out = drgg.moe_ffn_int8(X, logits, w1, s1, w2, s2, 1)
    few = torch.cat([torch.arange(5), torch.arange(T - 5, T)]).cuda()
    small = drgg.moe_ffn_int8(X[few], logits[few], w1, s1, w2, s2, 1)
    assert torch.equal(out[few], small)


# ---- the block ----------------------------------------------------------------------

def codes64(x):
    most = np.abs(x).max(1, keepdims=True) if x.size else np.zeros((len(x), 1))
    return np.rint(127 * x / np.where(most == 0, 1, most)), most[:, 0] / 127


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 64, 32), (9, 4, 4, 80, 48), (150, 6, 2, 256, 128), (600, 3, 2, 272, 144)])
def test_ffn_int8(drgg, T, E, k, H, I):
    """The block against 64 bits with the same quantisation.  A hidden value
    moved by rounding can take the next code (one step, about 1/40 of a row's
    rms, for a share of the codes below 1e-4), and the experts' outputs and
    the result are rounded to BF16: 2^-8 of the result's norm bounds the sum."""
    from dense_ragged_grouped_amd import moe
    rng = np.random.default_rng(T + E)
    X = dev(rng.standard_normal((T, H)).astype(np.float32), torch.bfloat16)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    W1q, s1 = moe.quantize_weights(dev((rng.standard_normal((E, 2 * I, H)) / np.sqrt(H)).astype(np.float32)))
    W2q, s2 = moe.quantize_weights(dev((rng.standard_normal((E, H, I)) / np.sqrt(I)).astype(np.float32)))
    got = host(moe.ffn_int8(X, dev(logits), W1q, s1, W2q, s2, k))
    w1, w2 = host(W1q).astype(np.float64) * host(s1)[..., None], host(W2q).astype(np.float64) * host(s2)[..., None]
    q, s = codes64(host(X))
    experts = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(logits.astype(np.float64), experts, 1)
    w = np.exp(top - top[:, :1])
    w /= w.sum(1, keepdims=True)
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            y = w1[experts[t, j]] @ q[t] * s[t]
            hq, hs = codes64((y[:I] / (1 + np.exp(-y[:I])) * y[I:])[None])
            want[t] += w[t, j] * (w2[experts[t, j]] @ hq[0] * hs[0])
    err = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert err < 2.0 ** -8, err


@pytest.mark.parametrize("T,E,k,H,I", [(0, 4, 2, 64, 32), (5, 8, 3, 96, 16), (700, 5, 2, 144, 272), (65, 1000, 20, 48, 16),
                                       (3, 300, 8, 4096, 32), (129, 130, 1, 4112, 16), (33000, 3, 1, 16, 16)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_ffn_is_its_operators(drgg, T, E, k, H, I, renormalize):
    """The one call gives the same bits as the operators called one by one, also on a side stream, into a given
    workspace full of garbage, and under graph replay."""
    rng = np.random.default_rng(T)
    X = dev(rng.standard_normal((T, H)).astype(np.float32), torch.bfloat16)
    logits = dev(rng.standard_normal((T, E)).astype(np.float32))
    w1, s1 = dev(rng.integers(-127, 128, (E, 2 * I, H)).astype(np.int8)), dev(rng.uniform(1, 2, (E, 2 * I)).astype(np.float32) / 999)
    w2, s2 = dev(rng.integers(-127, 128, (E, H, I)).astype(np.int8)), dev(rng.uniform(1, 2, (E, H)).astype(np.float32) / 999)
    r = drgg.moe_route(logits, k, renormalize=renormalize)
    q, s = drgg.quantize_int8(X, r.positions)
    h = drgg.grouped_gemm_int8(q, s, w1, s1, r.group_offsets, gated=True, out_dtype=torch.float32)
    q, s = drgg.quantize_int8(h)
    want = drgg.moe_combine(drgg.grouped_gemm_int8(q, s, w2, s2, r.group_offsets), r.positions, r.weights)
    args = (X, logits, w1, s1, w2, s2, k, renormalize)
    assert torch.equal(drgg.moe_ffn_int8(*args), want)
    ws = torch.full((drgg.ffn_workspace_size(T, E, k, H, I) + 16,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = [drgg.moe_ffn_int8(*args, workspace=ws, stream=side), drgg.moe_ffn_int8(*args, stream=side)]
    torch.cuda.synchronize()
    assert torch.equal(other[0], want) and torch.equal(other[1], want)
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(g):
        drgg.moe_ffn_int8(*args, workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        drgg.moe_ffn_int8(*args)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    if T:
        with pytest.raises(drgg.DrggError):
            drgg.moe_ffn_int8(*args, workspace=ws[:64])
        if H != I:   # else the transpose has the right shape
            with pytest.raises(ValueError):
                drgg.moe_ffn_int8(X, logits, w1, s1, w2.transpose(1, 2).contiguous(), s2, k)
        with pytest.raises(TypeError):
            drgg.moe_ffn_int8(X.float(), logits, w1, s1, w2, s2, k)


# ---- refusals --------------------------------------------------------------------------

def test_refusals(drgg):
    X, xs, W, ws = (dev(a) for a in operands(4, 32, 64, 2, 1))
    offsets = dev(np.array([0, 1, 4], np.int32))
    with pytest.raises(TypeError):
        drgg.grouped_gemm_int8(X.float(), xs, W, ws, offsets)
    with pytest.raises(TypeError):
        drgg.grouped_gemm_int8(X, xs.bfloat16(), W, ws, offsets)
    with pytest.raises(ValueError):
        drgg.grouped_gemm_int8(X, xs[:3], W, ws, offsets)
    with pytest.raises(ValueError):
        drgg.grouped_gemm_int8(X, xs, W, ws[:, :16].contiguous(), offsets)
    with pytest.raises(ValueError):
        drgg.grouped_gemm_int8(X, xs, W, ws, offsets[:2].contiguous())
    with pytest.raises(ValueError):
        drgg.grouped_gemm_int8(X, xs, W.transpose(1, 2), ws, offsets)
    with pytest.raises(ValueError):
        drgg.grouped_gemm_int8(X, xs, W, ws, offsets, out=torch.empty((4, 16), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        drgg.grouped_gemm_int8(X, xs, W, ws, offsets, out=torch.empty((4, 32), device="cuda"))
    with pytest.raises(drgg.DrggError):   # K not a multiple of 16
        drgg.gemm_int8(X[:, :40].contiguous(), xs, W[0, :, :40].contiguous(), ws[0].contiguous())
    with pytest.raises(drgg.DrggError):   # N not a multiple of 8, and of 16 when gated
        drgg.gemm_int8(X, xs, W[0, :20].contiguous(), ws[0, :20].contiguous())
    with pytest.raises(drgg.DrggError):
        drgg.gemm_int8(X, xs, W[0, :24].contiguous(), ws[0, :24].contiguous(), gated=True)
    with pytest.raises(drgg.DrggError):   # a sum that may not fit 32 bits
        drgg.gemm_int8(torch.zeros((1, 131072), dtype=torch.int8, device="cuda"), xs[:1].contiguous(),
                       torch.zeros((8, 131072), dtype=torch.int8, device="cuda"), ws[0, :8].contiguous())
    with pytest.raises(TypeError):
        drgg.grouped_gemm_int8(X, xs, W, ws, offsets, rows=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        drgg.gemm_int8(X, xs, W[0], ws[0], out_dtype=torch.float16)
    with pytest.raises(drgg.DrggError):
        drgg.quantize_int8(torch.zeros((2, 24), device="cuda"))
    with pytest.raises(TypeError):
        drgg.quantize_int8(torch.zeros((2, 32), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        drgg.quantize_int8(torch.zeros((2, 32), device="cuda"), torch.zeros((3, 2), dtype=torch.int32, device="cuda"))
    # the debug check of the offsets
    drgg.set_knob(drgg.KNOB_CHECK_OFFSETS, 1)
    try:
        drgg.grouped_gemm_int8(X, xs, W, ws, offsets)
        with pytest.raises(drgg.DrggError):
            drgg.grouped_gemm_int8(X, xs, W, ws, dev(np.array([0, 3, 2], np.int32)))
    finally:
        drgg.set_knob(drgg.KNOB_CHECK_OFFSETS, 0)
