"""The logits' gradient where masked experts' incoming gradients hold
infinities or NaN (their rows need not be finite): they take no part."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def drgg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as d
    return d


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("T,E,k", [(3, 4, 2), (70, 57, 5), (33, 300, 20)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_experts_take_no_part(drgg, T, E, k, renormalize, bad):
    """The same bits as with zeros in their place; zeros at every masked logit."""
    rng = np.random.default_rng(T)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[rng.random((T, E)) < 0.9] = -np.inf
    logits[::3] = -np.inf                       # tokens without any expert
    dw = rng.standard_normal((T, k)).astype(np.float32)
    l = torch.from_numpy(logits).cuda()
    r = drgg.moe_route(l, k, renormalize=renormalize)
    masked = np.isneginf(np.take_along_axis(logits, r.experts.cpu().numpy().astype(np.int64), 1))
    assert masked.any() and not masked.all()

    def grad(fill):
        d = torch.from_numpy(np.where(masked, np.float32(fill), dw)).cuda()
        return drgg.moe_route_grad(d, l, r.experts, r.weights, renormalize=renormalize)
    got = grad(bad)
    assert torch.equal(got, grad(0))
    got = got.cpu().numpy()
    assert not got[np.isneginf(logits)].any() and np.isfinite(got).all()
    # a lone expert's weight is 1 whatever its logit: something to check where a token has two
    assert got.any() == ((~masked).sum(1) > 1).any()


@pytest.mark.parametrize("renormalize", [True, False])
def test_live_experts_keep_their_nan(drgg, renormalize):
    l = torch.tensor([[1.0, 0.5, -np.inf, -np.inf], [1.0, 0.5, 0.25, -1.0]], device="cuda")
    r = drgg.moe_route(l, 2, renormalize=renormalize)
    d = torch.tensor([[np.nan, 1.0], [2.0, 1.0]], device="cuda")
    got = drgg.moe_route_grad(d, l, r.experts, r.weights, renormalize=renormalize).cpu().numpy()
    assert np.isnan(got[0, :2]).all() and not got[0, 2:].any() and np.isfinite(got[1]).all()
