"""The gradient of scored weights where it is small or nothing: one chosen
expert, one that has nearly all the weight, weights that a caller has changed.

Renormalised weights w_j = scale s_j / (sum of the chosen s) have, with f_j = 1 - s_j
(sigmoid) or 1 (softmax), the gradient w_j f_j (dw_j - r), r = sum_i w_i dw_i / scale.
One chosen expert has w = scale and so r = dw: exactly 0.  Where one has nearly all
the weight, dw_j - r is far below |dw_j| and has to keep its own precision.

Tolerance, u = 2^-24: with d_j = dw_j - dw_0, 0 the heaviest, the gradient is w_j f_j
(d_j - r), r = sum_i w_i d_i / scale.  A weight is within e = 2 (far + 20) u of itself
(tests/test_gpu_scores.py, far the distance of the exponents), d_j one rounding, f_j 6 u,
r e + (k + 4) u of its terms' magnitudes; with the last products, (2 e + (k + 16) u) of
w_j f_j (|d_j| + sum_i w_i |d_i| / scale).
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


def host(t):
    return t.cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


@pytest.mark.parametrize("T,E", [(1, 1), (1, 256), (5, 9), (700, 256), (33, 1000)])
@pytest.mark.parametrize("scale", [2.5, 1.7, 3.0, 1.0])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_one_chosen_expert_has_no_gradient(drgg, score, scale, T, E):
    from dense_ragged_grouped_amd import moe
    g = torch.Generator(device="cuda")
    g.manual_seed(T + E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    dw = torch.randn(T, 1, generator=g, device="cuda")
    sc = drgg.Scoring(score, bias=torch.randn(E, generator=g, device="cuda") * 0.01, scale=scale)
    r = drgg.moe_route_scores(logits, 1, sc)
    assert bool((r.weights == torch.tensor(scale, device="cuda")).all())
    assert not drgg.moe_route_scores_grad(dw, logits, r.experts, r.weights, sc).any()
    x = logits.requires_grad_()
    grad, = torch.autograd.grad(moe.route_scores(x, 1, sc).weights, x, dw)
    assert not grad.any()


@pytest.mark.parametrize("scale", [2.5, 1.7])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_one_chosen_expert_that_is_not_masked(drgg, score, scale):
    """The masked ones' weights are 0 and their dweights are not used."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    T, E, k = 300, 24, 3
    logits = torch.full((T, E), -float("inf"), device="cuda")
    logits[torch.arange(T), torch.randint(0, E, (T,), generator=g, device="cuda")] = torch.randn(T, generator=g, device="cuda")
    sc = drgg.Scoring(score, scale=scale)
    r = drgg.moe_route_scores(logits, k, sc)
    dw = torch.randn(T, k, generator=g, device="cuda")
    dw[r.weights == 0] = float("nan")
    assert not drgg.moe_route_scores_grad(dw, logits, r.experts, r.weights, sc).any()


def formula64(logits, dw, experts, w, score, scale):
    """(gradient at the chosen, the size that its error is relative to), from weights in 64 bits."""
    x = np.take_along_axis(logits, experts, 1)
    f = 1 / (1 + np.exp(x)) if score == "sigmoid" else np.ones_like(x)
    d = dw - np.take_along_axis(dw, w.argmax(1)[:, None], 1)
    r, size = ((w * v).sum(1, keepdims=True) / scale for v in (d, np.abs(d)))
    return w * f * (d - r), w * f * (np.abs(d) + size)


@pytest.mark.parametrize("k", [2, 3, 8, 17, 64])
@pytest.mark.parametrize("ahead", [3.0, 9.0, 16.0])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_one_expert_has_nearly_all_the_weight(drgg, score, ahead, k):
    T, E, scale = 200, 100, 2.5
    rng = np.random.default_rng(k)
    logits = rng.standard_normal((T, E)).astype(np.float32) - np.float32(4)
    logits[np.arange(T), rng.integers(0, E, T)] += np.float32(ahead)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    sc = drgg.Scoring(score, scale=scale)
    x = torch.from_numpy(logits).cuda()
    r = drgg.moe_route_scores(x, k, sc)
    got = host(drgg.moe_route_scores_grad(torch.from_numpy(dw).cuda(), x, r.experts, r.weights, sc))
    experts, l = host(r.experts).astype(np.int64), logits.astype(np.float64)
    log = np.take_along_axis(l if score == "softmax" else np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l))), experts, 1)
    far = (log.max(1, keepdims=True) - log).max(1, keepdims=True)
    w = np.exp(log - log.max(1, keepdims=True))
    want, size = formula64(l, dw.astype(np.float64), experts, scale * w / w.sum(1, keepdims=True), score, scale)
    tol = (4 * (far + 20) + k + 16) * U * size
    assert np.all(np.abs(np.take_along_axis(got, experts, 1) - want) <= tol)
    others = got.copy()
    np.put_along_axis(others, experts, 0, 1)
    assert not others.any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_weights_that_were_changed(drgg, score):
    """Weights that do not add up to the scale (pairs dropped after the selection): the formula with those weights, a
    weight of 0 as if not chosen.  Here dw_j - r is of the size of its terms: (k + 16) u of w_j f_j (|dw_j| + sum_i
    w_i |dw_i| / scale)."""
    T, E, k, scale = 300, 40, 5, 2.5
    rng = np.random.default_rng(11)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    sc = drgg.Scoring(score, scale=scale)
    x = torch.from_numpy(logits).cuda()
    r = drgg.moe_route_scores(x, k, sc)
    dropped = torch.from_numpy(rng.random((T, k)) < 0.4).cuda()
    weights = torch.where(dropped, torch.zeros_like(r.weights), r.weights)
    got = host(drgg.moe_route_scores_grad(torch.from_numpy(dw).cuda(), x, r.experts, weights, sc))
    experts, l, w, d = host(r.experts).astype(np.int64), logits.astype(np.float64), host(weights), dw.astype(np.float64)
    chosen = np.take_along_axis(l, experts, 1)
    f = 1 / (1 + np.exp(chosen)) if score == "sigmoid" else 1.0
    s, size = ((w * v).sum(1, keepdims=True) / scale for v in (d, np.abs(d)))
    tol = (k + 16) * U * w * f * (np.abs(d) + size)
    assert np.all(np.abs(np.take_along_axis(got, experts, 1) - w * f * (d - s)) <= tol)
