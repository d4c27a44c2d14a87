"""Calls of the 4-bit operators and the selection by scores at the ends of what they take: scales at either end of
the bytes' range against each other, rows with infinities and NaN through the serving block, as many chosen experts as
the lanes' slots hold.

Products of two elements are exact whatever the two scales are, and so are sums that fit 24 bits; else K roundings,
K 2^-24 of the sum of magnitudes.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_mxfp4 import U, block, host, operand  # noqa: E402
from tests.test_gpu_scores import choose, config, dev, make  # noqa: E402


@pytest.fixture(scope="module")
def drgg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as d
    import dense_ragged_grouped_amd.moe  # noqa: F401
    yield d
    d.set_knob(d.KNOB_TILE, 0)


@pytest.mark.parametrize("M,N,K", [(5, 24, 64), (300, 264, 320)])
@pytest.mark.parametrize("x,w", [((254, 254), (0, 0)), ((254, 254), (0, 3)), ((250, 254), (10, 12)), ((0, 0), (254, 254)),
                                 ((0, 2), (240, 254))])
def test_scales_far_apart(drgg, M, N, K, x, w):
    rng = np.random.default_rng(M)
    xc, xs, xv = operand(rng, M, K, lo=x[0], hi=x[1])
    wc, ws, wv = operand(rng, N, K, lo=w[0], hi=w[1])
    got = host(drgg.gemm_mxfp4(xc, xs, wc, ws, out_dtype=torch.float32))
    assert np.all(np.abs(got - xv @ wv.T) <= K * U * (np.abs(xv) @ np.abs(wv).T))


@pytest.mark.parametrize("tile", [0, 1, 2, 4])
@pytest.mark.parametrize("T,E,k,H,I", [(8, 8, 2, 64, 32), (130, 5, 3, 288, 160), (700, 8, 3, 544, 416)])
@pytest.mark.parametrize("scored", [False, True])
def test_block_with_infinities(drgg, scored, T, E, k, H, I, tile):
    """The block's result is its parts', NaN in the same places, and a bad row's NaN stay in its row."""
    from dense_ragged_grouped_amd import moe
    X, logits, bias, W1, W2 = block(drgg, T, E, H, I)
    sc = drgg.Scoring(bias=bias) if scored else None
    drgg.set_knob(drgg.KNOB_TILE, tile)
    w = (*moe.quantize_weights_mxfp4(W1), *moe.quantize_weights_mxfp4(W2))
    clean = drgg.moe_ffn_mxfp4(X, logits, *w, k, scoring=sc)
    X = X.clone()
    X[::5, 3], X[1::5, H - 1], X[2::5] = float("nan"), float("-inf"), 3e38
    got = drgg.moe_ffn_mxfp4(X, logits, *w, k, scoring=sc)
    r = drgg.moe_route_scores(logits, k, sc) if scored else drgg.moe_route(logits, k)
    h = drgg.grouped_gemm_mxfp4(*drgg.quantize_mxfp4(X), *w[:2], r.group_offsets, gated=True, rows=r.tokens,
                                out_dtype=torch.float32)
    y = drgg.grouped_gemm_mxfp4(*drgg.quantize_mxfp4(h), *w[2:], r.group_offsets)
    assert torch.equal(got.nan_to_num(5, 6, 7), drgg.moe_combine(y, r.positions, r.weights).nan_to_num(5, 6, 7))
    assert bool(got[::5].isnan().all()) and bool(got[1::5].isnan().all())
    for at in (3, 4):
        assert torch.equal(got[at::5], clean[at::5])


@pytest.mark.parametrize("kind", ["close", "ties", "bias", "masked"])
@pytest.mark.parametrize("k", [15, 16, 32, 47, 48, 63])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_slots_filled_by_the_chosen(drgg, score, k, kind):
    """Sixteen lanes hold the chosen in slots: the gap behind the last one lies in the next slot, or in none."""
    logits, bias = make(kind, 70, 64, k)
    for groups in (1, 2, 4, 8):
        c = config(score, groups, groups)
        r = drgg.moe_route_scores(dev(logits), k, drgg.Scoring(**c, bias=None if bias is None else dev(bias)))
        assert np.array_equal(host(r.experts), choose(logits, bias, c, k)[0])
