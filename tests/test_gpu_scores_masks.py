"""Groups of experts where biases are far from the scores: finite masks (-1e9,
the type's lowest value), pairs that cancel.  The groups are those of 64-bit values;
and a mask on experts that nobody chooses does not send the tokens through 64 bits.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_scores import choose, config, dev, host, scores64  # noqa: E402

LOWEST = np.finfo(np.float32).min


@pytest.fixture(scope="module")
def drgg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as d
    return d


def biases(kind, E, groups, rng):
    b = (np.round(rng.standard_normal(E) * 30) * 0.001).astype(np.float32)
    size = E // groups
    if kind == "one":
        b[rng.integers(E)] = -1e9
    elif kind == "group":
        b[size:2 * size] = -1e9
    elif kind == "half":
        b[rng.random(E) < 0.5] = -1e6
    elif kind == "lowest":
        b[rng.random(E) < 0.3] = LOWEST
    elif kind == "lowest groups":   # sums of two leave FP32's range, of two groups by as much
        b[size:3 * size] = LOWEST
        b[3 * size:] = -np.inf
    elif kind == "mixed":
        b = np.where(rng.random(E) < 0.5, b, np.sign(b) * np.exp2(rng.uniform(-10, 40, E))).astype(np.float32)
    return b


@pytest.mark.parametrize("kind", ["one", "group", "half", "lowest", "lowest groups", "mixed"])
@pytest.mark.parametrize("T,E,k,groups,top", [(130, 256, 8, 8, 4), (67, 100, 6, 4, 2), (70, 64, 4, 32, 9), (65, 1024, 8, 16, 5),
                                              (66, 48, 3, 16, 4), (64, 32, 4, 8, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_choice(drgg, score, T, E, k, groups, top, kind):
    rng = np.random.default_rng(T + E)
    logits, bias = rng.standard_normal((T, E)).astype(np.float32), biases(kind, E, groups, rng)
    for best in (1, 2):
        c = config(score, groups, top, best)
        r = drgg.moe_route_scores(dev(logits), k, drgg.Scoring(**c, bias=dev(bias)))
        assert np.array_equal(host(r.experts), choose(logits, bias, c, k)[0]), best


def cancelling(score, size):
    """Two groups of equal value but for their scores: 96 twice, and 1e9 with 192 - 1e9."""
    rng = np.random.default_rng(size)
    E = 4 * size
    logits = rng.standard_normal((200, E)).astype(np.float32)
    bias = np.full(E, -3e9, np.float32)
    bias[:2] = 96
    bias[size:size + 2] = 1e9, -1e9 + 192
    bias[2 * size:] = 0
    return logits, bias


@pytest.mark.parametrize("size", [4, 25, 32])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_values_that_cancel(drgg, score, size):
    logits, bias = cancelling(score, size)
    c = config(score, 4, 1)
    want = choose(logits, bias, c, 2)[0]
    v32 = scores64(logits, score).astype(np.float32) + bias
    first = v32[:, 0] + v32[:, 1] >= v32[:, size] + v32[:, size + 1]
    assert (first != (want[:, 0] < size)).any() and 20 < (want[:, 0] < size).sum() < 180   # FP32 does not decide
    r = drgg.moe_route_scores(dev(logits), 2, drgg.Scoring(**c, bias=dev(bias)))
    assert np.array_equal(host(r.experts), want)


@pytest.mark.parametrize("groups,E", [(8, 256), (8, 160)])
@pytest.mark.parametrize("mask", [-1e6, -1e9, float(LOWEST)])
def test_masked_experts_cost_no_more_than_infinite_ones(drgg, mask, E, groups):
    """By the wide margin that a bias of -1e6 and less gives, every token was chosen again: 3.3 times the time of a bias of
    -inf; by the groups' own errors 1.1 times.  Medians of calls in turn."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    logits = torch.randn(16384, E, generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") * 0.03
    times = {}
    drgg.set_knob(drgg.KNOB_TIMING, 1)
    try:
        for _ in range(12):
            for value in (mask, -float("inf")):
                b = bias.clone()
                b[77], b[E // groups:2 * (E // groups)] = value, value
                drgg.moe_route_scores(logits, 8, drgg.Scoring(bias=b, groups=groups, top_groups=4))
                times.setdefault(value, []).append(dict(drgg.last_call_kernel_times())["moe_select_scores_kernel"])
    finally:
        drgg.set_knob(drgg.KNOB_TIMING, 0)
    finite, infinite = (sorted(t)[len(t) // 2] for t in times.values())
    assert finite < 1.7 * infinite
