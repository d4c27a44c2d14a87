"""Microscaled 4-bit floating point on the GPU: quantisation, products and the
serving block, against plain implementations in 64 bits (NumPy).

Tolerances, u = 2^-24:
* Codes, scales and dequantised values: equal.
* Products of two elements are exact, and so is their sum where it fits 24 bits
  (scales in a narrow range): equal in FP32, and in BF16 the one rounding.  With
  wide scales K roundings in any order: K u of the sum of magnitudes.
* The gate: (4 |g| + 16) u of the result, and 0 for its value below g = -87.
* BF16: half a step, 2^-8 of the value's power of two.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
TABLE = np.concatenate([VALUES, -VALUES])


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


def step(v, dtype):
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    return half * np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))))


# ---- the format in 64 bits --------------------------------------------------------

def quantize64(x):
    """(codes [T, K], one a byte, scale bytes [T, K/32]) by distance to every code."""
    T, K = x.shape
    b = x.astype(np.float64).reshape(T, K // 32, 32)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[:, :, None], 0.0, b)
    most = np.abs(b).max(2)
    with np.errstate(divide="ignore"):
        byte = np.where(most == 0, 0, np.clip(np.floor(np.log2(np.where(most == 0, 1, most))) - 2 + 127, 0, 254)).astype(int)
    a = np.abs(b) * np.exp2(127.0 - byte)[:, :, None]
    near = np.abs(a[..., None] - VALUES)
    least = near.min(-1, keepdims=True)
    code = np.where(near == least, np.arange(8) % 2 * 8 + np.arange(8), 99).argmin(-1)   # an even one among two as near
    code = code + 8 * np.signbit(np.where(bad[:, :, None], 0.0, b))
    return code.reshape(T, K).astype(np.uint8), np.where(bad, 255, byte).astype(np.uint8)


def pack(codes):
    return codes[..., 0::2] | codes[..., 1::2] << 4


def lay(scales, fill=0):
    """[.., rows, K/32] to [ceil(K/256), .., rows, 8], `fill` past the row's end."""
    n = -scales.shape[-1] % 8
    padded = np.concatenate([scales, np.full((*scales.shape[:-1], n), fill, np.uint8)], -1)
    return np.ascontiguousarray(np.moveaxis(padded.reshape(*scales.shape[:-1], -1, 8), -2, 0))


def values(codes, scales):
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return TABLE[codes] * np.repeat(s, 32, -1)


def operand(rng, *shape, lo=125, hi=129, fill=0):
    """(codes and scales on the device, the values)"""
    codes = rng.integers(0, 16, shape, dtype=np.uint8)
    scales = rng.integers(lo, hi + 1, (*shape[:-1], shape[-1] // 32), dtype=np.uint8)
    return dev(pack(codes)), dev(lay(scales, fill)), values(codes, scales)


# ---- quantisation -------------------------------------------------------------------

def make(kind, T, K, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, K)).astype(np.float32)
    if kind == "spread":
        x *= np.exp2(rng.integers(-140, 120, (T, K // 32)).astype(np.float32)).repeat(32, 1)
    elif kind == "ties":   # borders between codes, exactly and one step beside
        x = rng.choice(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7, 0, 4], np.float32), (T, K))
        x[:, ::32] = 4
        x = np.where(rng.random((T, K)) < 0.3, np.nextafter(x, np.float32(0)), x)
        x = np.where(rng.random((T, K)) < 0.5, -x, x).astype(np.float32)
    elif kind == "edges":
        x *= np.float32(1e-41)
        x[0::5] = 0
        x[1::5, :40] = np.inf
        x[2::5, K // 2] = np.nan
        x[3::5] = np.finfo(np.float32).max
        x[4::5] = np.where(rng.random(x[4::5].shape) < 0.5, np.float32(2.0 ** -126), np.float32(3e38))
    return x


@pytest.mark.parametrize("kind", ["normal", "spread", "ties", "edges"])
@pytest.mark.parametrize("T,K", [(1, 32), (5, 64), (17, 224), (3, 256), (9, 288), (130, 2048), (2, 4128), (1025, 96)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize(drgg, T, K, kind, dtype):
    x = dev(make(kind, T, K, T + K)).to(dtype)
    codes, scales = drgg.quantize_mxfp4(x)
    want, byte = quantize64(host(x))
    assert np.array_equal(host(scales), lay(byte))
    assert np.array_equal(host(codes), pack(want))
    v = values(want, byte)
    for out in (torch.float32, torch.bfloat16):
        got = host(drgg.dequantize_mxfp4(codes, scales, dtype=out))
        assert np.array_equal(np.isnan(got), np.isnan(v))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(v))


def test_dequantize_all(drgg):
    """Every code under every scale byte; what is past the type's range is infinite."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    v = values(codes, scales)
    for dtype, most in ((torch.float32, 2.0 ** 128), (torch.bfloat16, 2.0 ** 128)):
        got = host(drgg.dequantize_mxfp4(dev(pack(codes)), dev(lay(scales)), dtype=dtype))
        want = np.where(np.abs(v) >= most, np.sign(v) * np.inf, v)
        assert np.array_equal(got, want, equal_nan=True)


def test_scales_layout(drgg):
    rng = np.random.default_rng(0)
    s = rng.integers(0, 256, (3, 5, 19), dtype=np.uint8)
    assert np.array_equal(host(drgg.mxfp4_scales(dev(s))), lay(s))


def test_no_rows(drgg):
    codes, scales = drgg.quantize_mxfp4(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 32) and scales.shape == (1, 0, 8)
    assert drgg.dequantize_mxfp4(codes, scales).shape == (0, 64)


# ---- products -----------------------------------------------------------------------

def grouped64(x, w, offsets, N):
    y, mag = np.zeros((x.shape[0], N)), np.zeros((x.shape[0], N))
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        y[lo:hi] = x[lo:hi] @ w[e].T
        mag[lo:hi] = np.abs(x[lo:hi]) @ np.abs(w[e]).T
    return y, mag


def gate64(y):
    I = y.shape[1] // 2
    g, u = y[:, :I], y[:, I:]
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u, g


def check(got, want, g=None, slack=0.0):
    tol = step(want, got.dtype) + slack
    if g is not None:
        tol = tol + 1.01 * (4 * np.abs(g) + 16) * U * np.abs(want)
        tol = np.where(g < -87, np.abs(want) * 1.01 + tol, tol)
    assert np.all(np.abs(host(got) - want) <= tol)


def counts_to_offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


GROUPED = [([1], 8, 32), ([3], 16, 64), ([0, 5, 0], 24, 96), ([17, 1, 33, 0, 64, 65], 200, 288), ([700], 264, 1056),
           ([130, 0, 257, 3], 144, 512), ([1] * 40, 72, 736), ([64] * 8, 1536, 256), ([300, 20], 520, 2048),
           ([513, 255], 776, 160), ([2000, 1500, 3], 256, 384), ([0] * 1000 + [7] * 24, 32, 128)]


@pytest.mark.parametrize("counts,N,K", GROUPED)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_exact(drgg, counts, N, K, dtype, gated):
    """Sums that fit 24 bits are exact; the bytes past a row's last scale hold anything but 255."""
    rng = np.random.default_rng(N + K)
    N = 2 * N if gated else N
    E, M = len(counts), sum(counts)
    x, xs, xv = operand(rng, M, K, fill=254)
    w, ws, wv = operand(rng, E, N, K, fill=254)
    offsets = counts_to_offsets(counts)
    y, mag = grouped64(xv, wv, offsets, N)
    assert mag.max() * 64 < 2 ** 24   # multiples of (2^-2 * 0.5)^2
    got = drgg.grouped_gemm_mxfp4(x, xs, w, ws, dev(offsets), gated=gated, out_dtype=dtype)
    if gated:
        check(got, *gate64(y))
    else:
        assert torch.equal(got, dev(y).to(torch.float32).to(dtype))


@pytest.mark.parametrize("counts,N,K", [([33, 5], 72, 736), ([700], 264, 1056), ([300, 0, 20], 520, 2048)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_wide_scales(drgg, counts, N, K, dtype):
    rng = np.random.default_rng(N + K + 1)
    x, xs, xv = operand(rng, sum(counts), K, lo=100, hi=150)
    w, ws, wv = operand(rng, len(counts), N, K, lo=100, hi=150)
    offsets = counts_to_offsets(counts)
    y, mag = grouped64(xv, wv, offsets, N)
    got = drgg.grouped_gemm_mxfp4(x, xs, w, ws, dev(offsets), out_dtype=dtype)
    check(got, y, slack=K * U * mag)


@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 4096, 4096), (16, 256, 2048), (100, 136, 4128), (300, 1000, 992)])
@pytest.mark.parametrize("gated", [False, True])
def test_dense(drgg, M, N, K, gated):
    rng = np.random.default_rng(M + N)
    N = 2 * N if gated else N
    x, xs, xv = operand(rng, M, K)
    w, ws, wv = operand(rng, N, K)
    y = xv @ wv.T
    for dtype in (torch.float32, torch.bfloat16):
        got = drgg.gemm_mxfp4(x, xs, w, ws, gated=gated, out_dtype=dtype)
        if gated:
            check(got, *gate64(y))
        else:
            assert torch.equal(got, dev(y).to(torch.float32).to(dtype))


@pytest.mark.parametrize("counts,T,N,K", [([3, 0, 20], 9, 40, 96), ([300, 40, 333], 100, 272, 544), ([5] * 30, 7, 64, 1056),
                                          ([900, 1100], 1500, 528, 256)])
@pytest.mark.parametrize("gated", [False, True])
def test_gathered(drgg, counts, T, N, K, gated):
    """Rows by index, some named often, some outside the rows, which read as zeros."""
    rng = np.random.default_rng(T)
    N = 2 * N if gated else N
    M = sum(counts)
    x, xs, xv = operand(rng, T, K)
    w, ws, wv = operand(rng, len(counts), N, K)
    offsets = counts_to_offsets(counts)
    rows = rng.integers(0, T, M).astype(np.int32)
    rows[::7] = [-1, T, 2 ** 31 - 1, -2 ** 31][M % 4]
    inside = (rows >= 0) & (rows < T)
    picked = np.where(inside[:, None], xv[np.where(inside, rows, 0)], 0)
    y, _ = grouped64(picked, wv, offsets, N)
    for dtype in (torch.float32, torch.bfloat16):
        got = drgg.grouped_gemm_mxfp4(x, xs, w, ws, dev(offsets), gated=gated, rows=dev(rows), out_dtype=dtype)
        if gated:
            check(got, *gate64(y))
        else:
            assert torch.equal(got, dev(y).to(torch.float32).to(dtype))


TILES = [1, 2, 4]   # 256x256, 128x128, 128x256


@pytest.fixture
def forced(drgg):
    def force(tile):
        drgg.set_knob(drgg.KNOB_TILE, tile)
    yield force
    drgg.set_knob(drgg.KNOB_TILE, 0)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("counts,N,K", [([1], 8, 32), ([3, 0, 300], 136, 96), ([17, 1, 33, 0, 64, 265], 264, 288),
                                        ([513, 255, 0, 130], 520, 1056), ([700], 1000, 736), ([40] * 30, 72, 128),
                                        ([5] * 1000, 32, 64), ([2100, 900], 776, 160), ([256], 256, 4096)])
@pytest.mark.parametrize("gated,gathered", [(False, False), (True, False), (False, True), (True, True)])
def test_every_tile(drgg, forced, tile, counts, N, K, gated, gathered):
    """The tiles, whatever the rule would take: several per workgroup, cut at every edge, K within one stage and past
    whole ones, the bytes past a row's last scale not 0."""
    rng = np.random.default_rng(N + K)
    N = 2 * N if gated else N
    E, M = len(counts), sum(counts)
    T = M // 2 + 3 if gathered else M
    x, xs, xv = operand(rng, T, K, fill=254)
    w, ws, wv = operand(rng, E, N, K, fill=254)
    offsets = counts_to_offsets(counts)
    rows = None
    if gathered:
        rows = rng.integers(0, T, M).astype(np.int32)
        rows[::11] = T
        xv = np.where((rows < T)[:, None], xv[np.minimum(rows, T - 1)], 0)
        rows = dev(rows)
    y, mag = grouped64(xv, wv, offsets, N)
    assert mag.max() * 64 < 2 ** 24
    forced(tile)
    for dtype in (torch.float32, torch.bfloat16):
        got = drgg.grouped_gemm_mxfp4(x, xs, w, ws, dev(offsets), gated=gated, rows=rows, out_dtype=dtype)
        if gated:
            check(got, *gate64(y))
        else:
            assert torch.equal(got, dev(y).to(torch.float32).to(dtype))


@pytest.mark.parametrize("M,N", [(20, 72), (700, 264)])
def test_nan_scales_stay_in_their_row_and_column(drgg, M, N):
    rng = np.random.default_rng(2)
    K = 320
    xc, wc = rng.integers(0, 16, (M, K), dtype=np.uint8), rng.integers(0, 16, (N, K), dtype=np.uint8)
    sx, sw = np.full((M, K // 32), 127, np.uint8), np.full((N, K // 32), 126, np.uint8)
    sx[3, 9], sw[11, 0] = 255, 255
    got = host(drgg.gemm_mxfp4(dev(pack(xc)), dev(lay(sx)), dev(pack(wc)), dev(lay(sw)), out_dtype=torch.float32))
    bad = np.zeros((M, N), bool)
    bad[3], bad[:, 11] = True, True
    assert np.array_equal(np.isnan(got), bad)
    y = values(xc, np.where(sx == 255, 0, sx)) @ values(wc, np.where(sw == 255, 0, sw)).T
    assert np.array_equal(got[~bad], y[~bad])


@pytest.mark.parametrize("counts", [[4, 3], [400, 300]])
def test_rows_outside_the_groups_are_left(drgg, counts):
    rng = np.random.default_rng(5)
    M, N, K = sum(counts) + 6, 72, 128
    x, xs, xv = operand(rng, M, K)
    w, ws, wv = operand(rng, 2, N, K)
    offsets = counts_to_offsets(counts)
    out = torch.full((M, N), 7.0, device="cuda")
    drgg.grouped_gemm_mxfp4(x, xs, w, ws, dev(offsets), out_dtype=torch.float32, out=out)
    y, _ = grouped64(xv, wv, offsets, N)
    assert np.array_equal(host(out)[:M - 6], y[:M - 6]) and bool((out[M - 6:] == 7).all())


def test_small_scales(drgg):
    """Results below FP32's normal range keep their value to its smallest step, and large ones overflow to infinity."""
    rng = np.random.default_rng(6)
    x, xs, xv = operand(rng, 20, 64, lo=60, hi=64)
    w, ws, wv = operand(rng, 24, 64, lo=60, hi=64)
    y = xv @ wv.T
    got = host(drgg.gemm_mxfp4(x, xs, w, ws, out_dtype=torch.float32))
    assert np.all(np.abs(got - y) <= 64 * U * (np.abs(xv) @ np.abs(wv).T) + 64 * 2.0 ** -126)
    x, xs, xv = operand(rng, 20, 64, lo=200, hi=200)
    w, ws, wv = operand(rng, 24, 64, lo=200, hi=200)
    y = xv @ wv.T
    got = host(drgg.gemm_mxfp4(x, xs, w, ws, out_dtype=torch.float32))
    assert np.isinf(got[np.abs(y) > 2.0 ** 129]).all()


# ---- the serving block -----------------------------------------------------------------

def block(drgg, T, E, H, I, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    X, logits, bias = normal(T, H), normal(T, E, dtype=torch.float32), normal(E, dtype=torch.float32) * 0.01
    return X, logits, bias, normal(E, 2 * I, H) * 0.05, normal(E, H, I) * 0.05


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 64, 32), (8, 32, 4, 2048, 768), (130, 5, 3, 288, 160), (1500, 8, 3, 544, 416)])
@pytest.mark.parametrize("scored", [False, True])
def test_ffn_is_its_parts(drgg, T, E, k, H, I, scored):
    ffn_is_its_parts(drgg, T, E, k, H, I, scored)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("T,E,k,H,I", [(40, 3, 2, 96, 32), (300, 5, 3, 288, 160), (900, 2, 2, 544, 416), (700, 40, 1, 64, 352)])
def test_ffn_is_its_parts_in_every_tile(drgg, forced, tile, T, E, k, H, I):
    """The activation's codes and scales are made in the first product's epilogue: their bytes past a row's end have to
    be written too, whatever the workspace held."""
    forced(tile)
    ffn_is_its_parts(drgg, T, E, k, H, I, True)


def ffn_is_its_parts(drgg, T, E, k, H, I, scored):
    from dense_ragged_grouped_amd import moe
    X, logits, bias, W1, W2 = block(drgg, T, E, H, I)
    w1, s1 = moe.quantize_weights_mxfp4(W1)
    w2, s2 = moe.quantize_weights_mxfp4(W2)
    sc = drgg.Scoring(bias=bias, scale=2.5) if scored else None
    dirty = torch.full((drgg.ffn_mxfp4_workspace_size(T, E, k, H, I),), 255, dtype=torch.uint8, device="cuda")
    got = drgg.moe_ffn_mxfp4(X, logits, w1, s1, w2, s2, k, scoring=sc, workspace=dirty)
    assert torch.equal(got, moe.ffn_mxfp4(X, logits, w1, s1, w2, s2, k, scoring=sc))
    r = drgg.moe_route_scores(logits, k, sc) if scored else drgg.moe_route(logits, k)
    x, xs = drgg.quantize_mxfp4(X)
    h = drgg.grouped_gemm_mxfp4(x, xs, w1, s1, r.group_offsets, gated=True, rows=r.tokens, out_dtype=torch.float32)
    y = drgg.grouped_gemm_mxfp4(*drgg.quantize_mxfp4(h), w2, s2, r.group_offsets)
    assert torch.equal(got, drgg.moe_combine(y, r.positions, r.weights))


def test_ffn_against_64_bits(drgg):
    """Two BF16 roundings, 2^-8 each; an activation near the border of two codes may take the other one (0.2 % of the
    norm allowed for all of them: one in some thousand values, by half a block's largest, would make 0.1 %)."""
    from dense_ragged_grouped_amd import moe
    T, E, k, H, I = 200, 8, 3, 544, 416
    X, logits, bias, W1, W2 = block(drgg, T, E, H, I, 1)
    w1, s1 = moe.quantize_weights_mxfp4(W1)
    w2, s2 = moe.quantize_weights_mxfp4(W2)
    r = drgg.moe_route_scores(logits, k, drgg.Scoring(bias=bias))
    got = host(moe.ffn_mxfp4(X, logits, w1, s1, w2, s2, k, scoring=drgg.Scoring(bias=bias)))

    def rounded(x):
        return values(*quantize64(x))
    w1v, w2v = rounded(host(W1).reshape(-1, H)).reshape(E, 2 * I, H), rounded(host(W2).reshape(-1, I)).reshape(E, H, I)
    xv, want = rounded(host(X)), np.zeros((T, H))
    for t in range(T):
        for e, w in zip(host(r.experts)[t], host(r.weights)[t]):
            h, _ = gate64((w1v[e] @ xv[t])[None])
            want[t] += w * (w2v[e] @ rounded(h)[0])
    assert np.linalg.norm(got - want) <= (2 * 2.0 ** -8 + 0.002) * np.linalg.norm(want)


# ---- calls ---------------------------------------------------------------------------

def test_refusals(drgg):
    x, xs = drgg.quantize_mxfp4(torch.randn(6, 64, device="cuda"))
    w, ws = (t.view(*s) for t, s in zip(drgg.quantize_mxfp4(torch.randn(32, 64, device="cuda")), ((2, 16, 32), (1, 2, 16, 8))))
    o = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    for bad in (lambda: drgg.quantize_mxfp4(torch.randn(4, 48, device="cuda")),
                lambda: drgg.quantize_mxfp4(torch.randn(4, 64, device="cuda").half()),
                lambda: drgg.quantize_mxfp4(torch.randn(4, 128, device="cuda")[:, ::2]),
                lambda: drgg.quantize_mxfp4(torch.randn(4, 64)),
                lambda: drgg.dequantize_mxfp4(x, xs[:, :5].contiguous()),
                lambda: drgg.dequantize_mxfp4(x.to(torch.int8), xs),
                lambda: drgg.dequantize_mxfp4(x, xs, dtype=torch.float16),
                lambda: drgg.grouped_gemm_mxfp4(x, xs, w[:1], ws[:, :1].contiguous(), o),
                lambda: drgg.grouped_gemm_mxfp4(x[:, :16].contiguous(), xs, w, ws, o),
                lambda: drgg.grouped_gemm_mxfp4(x, xs, w, ws.view(1, 32, 8), o),
                lambda: drgg.grouped_gemm_mxfp4(x, xs, w[:, :12].contiguous(), ws[:, :, :12].contiguous(), o),
                lambda: drgg.grouped_gemm_mxfp4(x, xs, w[:, :8].contiguous(), ws[:, :, :8].contiguous(), o, gated=True),
                lambda: drgg.gemm_mxfp4(x, xs, w[0], ws[:, 0].contiguous(), out=torch.empty(6, 15, device="cuda").bfloat16())):
        with pytest.raises((TypeError, ValueError, drgg.DrggError)):
            bad()


def test_captured_on_a_forked_stream(drgg):
    """The block in two graphs, replayed in turn on changing rows beside eager calls."""
    from dense_ragged_grouped_amd import moe
    made = []
    for T in (8, 300):
        X, logits, bias, W1, W2 = block(drgg, T, 8, 256, 96, T)
        w = (*moe.quantize_weights_mxfp4(W1), *moe.quantize_weights_mxfp4(W2))
        sc = drgg.Scoring(bias=bias)

        def call(stream=None, X=X, logits=logits, w=w, sc=sc):
            return drgg.moe_ffn_mxfp4(X, logits, *w, 2, scoring=sc, stream=stream)
        call()
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            out = call(side)
            torch.cuda.current_stream().wait_stream(side)
        made.append((X, logits, call, graph, out))
    for _ in range(3):
        for X, logits, call, graph, out in made:
            X.copy_(torch.randn_like(X))
            logits.copy_(torch.randn_like(logits))
            graph.replay()
            assert torch.equal(out, call())
            torch.cuda.synchronize()


def test_two_calls_on_two_streams(drgg):
    from dense_ragged_grouped_amd import moe
    X, logits, bias, W1, W2 = block(drgg, 400, 8, 256, 96)
    w = (*moe.quantize_weights_mxfp4(W1), *moe.quantize_weights_mxfp4(W2))
    want = [drgg.moe_ffn_mxfp4(X, logits, *w, 2), drgg.moe_ffn_mxfp4(X.flip(0), logits, *w, 2)]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    flipped = X.flip(0)
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [drgg.moe_ffn_mxfp4(x, logits, *w, 2, stream=s) for x, s in zip((X, flipped), sides)]
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
