"""Second derivatives through the differentiable operators: their backward
passes run in kernels that autograd cannot see into, so a second derivative has
to raise an error, never to come back without the part that passes through
them.  Runs on the CPU with torch's products in the kernels' place; float64,
small integers, so first derivatives are compared exactly."""
import pytest

torch = pytest.importorskip("torch")

from dense_ragged_grouped_amd import Routing, autograd, moe

ASK = "second derivative"


def rand(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-4, 5, shape, generator=g).double().requires_grad_(True)


def plain_route(logits, k, renormalize=True):
    top, experts = torch.topk(logits, k, dim=1)
    order = experts.flatten().argsort(stable=True)
    positions = torch.empty_like(order)
    positions[order] = torch.arange(order.numel())
    offsets = torch.searchsorted(experts.flatten()[order], torch.arange(logits.shape[1] + 1))
    return Routing(experts, torch.softmax(top, 1), offsets, positions.view_as(experts), order // k)


def plain_route_grad(dw, logits, experts, w, renormalize=True):
    return torch.zeros_like(logits).scatter(1, experts, w * (dw - (w * dw).sum(1, keepdim=True)))


def plain_dispatch(X, positions):
    out = X.new_empty((positions.numel(), X.shape[1]))
    out[positions.flatten()] = X.repeat_interleave(positions.shape[1], 0)
    return out


def plain_combine(rows, positions, weights=None):
    picked = rows[positions]
    return (picked if weights is None else picked * weights[..., None]).sum(1)


def plain_combine_grad(dout, rows, positions, weights):
    drows = torch.empty_like(rows)
    drows[positions.flatten()] = (weights[..., None] * dout[:, None, :]).flatten(0, 1)
    return drows, (rows[positions] * dout[:, None, :]).sum(2)


def per_group(fn, offsets):
    return [fn(e, slice(int(offsets[e]), int(offsets[e + 1]))) for e in range(len(offsets) - 1)]


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    for name, fn in (("moe_route", plain_route), ("moe_route_grad", plain_route_grad), ("moe_dispatch", plain_dispatch),
                     ("moe_combine", plain_combine), ("moe_combine_grad", plain_combine_grad)):
        monkeypatch.setattr(moe, name, fn)
    monkeypatch.setattr(autograd, "grouped_gemm_fwd", lambda X, W, o, out_dtype: torch.cat(
        per_group(lambda e, s: X[s] @ W[e].t(), o)))
    monkeypatch.setattr(autograd, "grouped_gemm_dgrad", lambda G, W, o, out_dtype: torch.cat(
        per_group(lambda e, s: G[s] @ W[e], o)))
    monkeypatch.setattr(autograd, "grouped_gemm_wgrad", lambda X, G, o, out_dtype, deterministic: torch.stack(
        per_group(lambda e, s: G[s].t() @ X[s], o)))


POSITIONS = torch.tensor([[0, 3], [4, 1], [2, 5]])
OFFSETS = torch.tensor([0, 2, 2, 5], dtype=torch.int32)


def cases():
    """name -> (function, its inputs, the same from torch operations)"""
    return {
        "route": (lambda l: moe.route(l, 2).weights, (torch.linspace(-1, 1, 12, dtype=torch.float64).view(3, 4)
                                                      .requires_grad_(True),),
                  lambda l: torch.softmax(torch.topk(l, 2, dim=1)[0], 1)),
        "dispatch": (lambda x: moe.dispatch(x, POSITIONS), (rand(3, 5),),
                     lambda x: torch.index_select(x, 0, POSITIONS.flatten().argsort() // 2)),
        "combine": (lambda r, w: moe.combine(r, POSITIONS, w), (rand(6, 5), rand(3, 2, seed=1)),
                    lambda r, w: (r[POSITIONS] * w[..., None]).sum(1)),
        "grouped_linear": (lambda x, w: autograd.grouped_linear(x, w, OFFSETS), (rand(5, 4), rand(3, 2, 4, seed=1)),
                           lambda x, w: torch.cat(per_group(lambda e, s: x[s] @ w[e].t(), OFFSETS))),
    }


@pytest.mark.parametrize("name", sorted(cases()))
@pytest.mark.parametrize("create_graph", [False, True])
def test_first_derivatives(name, create_graph):
    fn, inputs, plain = cases()[name]
    got = torch.autograd.grad(fn(*inputs).pow(2).sum(), inputs, create_graph=create_graph)
    want = torch.autograd.grad(plain(*inputs).pow(2).sum(), inputs)
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("name", sorted(cases()))
@pytest.mark.parametrize("loss", ["linear", "square"])
def test_second_derivatives_raise(name, loss):
    """Also where the incoming gradient is a constant (a linear loss), and where only one input is asked for: the
    plain form's second derivative tells which inputs there is one for."""
    fn, inputs, plain = cases()[name]

    def penalty(f):
        y = f(*inputs)
        first = torch.autograd.grad(y.sum() if loss == "linear" else y.pow(2).sum(), inputs, create_graph=True)
        return sum((g * torch.arange(1, g.numel() + 1).view_as(g)).pow(2).sum() for g in first)
    p = penalty(plain)
    if not p.requires_grad:   # a linear loss of a linear operator
        assert name == "dispatch"
        return
    want = torch.autograd.grad(p, inputs, allow_unused=True)
    assert any(w is not None for w in want)
    for x, w in zip(inputs, want):
        if w is not None and bool(w.any()):
            with pytest.raises(RuntimeError, match=ASK):
                torch.autograd.grad(penalty(fn), x)
    with pytest.raises(RuntimeError, match=ASK):
        penalty(fn).backward()


def test_second_derivative_past_the_operators(monkeypatch):
    """A graph kept for another part's second derivative stays usable."""
    r, w = rand(6, 5), rand(3, 2, seed=1)
    a = rand(3, 5, seed=2)
    loss = (moe.combine(r, POSITIONS, w) + a ** 3).sum()
    dr, da = torch.autograd.grad(loss, (r, a), create_graph=True)
    assert torch.equal(torch.autograd.grad(da.sum(), a)[0], 6 * a)


def test_saved_by_hooks():
    """grouped_linear hands its tensors to active saved-tensor hooks, which keep no graph: the backward itself raises
    when a graph of it is asked for, and works without."""
    x, w = rand(5, 4), rand(3, 2, 4, seed=1)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), lambda t: t):
        y = autograd.grouped_linear(x, w, OFFSETS)
    torch.autograd.grad(y.sum(), (x, w), retain_graph=True)
    with pytest.raises(RuntimeError, match=ASK):
        torch.autograd.grad(y.sum(), (x, w), create_graph=True)
