"""Calls with stream= on the GPU: the results' memory belongs to the stream
that writes them, and their values are those of a call on the current stream."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def drgg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as d
    return d


def home_stream(t):
    """The handle of the stream whose memory holds t."""
    at = t.data_ptr()
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= at < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not the allocator's memory")


def calls(d):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    T, E, k, H, N = 130, 4, 2, 64, 96
    X, G, W = normal(T * k, H), normal(T * k, N), normal(E, N, H)
    logits, dw, dout = normal(T, E, dtype=torch.float32), normal(T, k, dtype=torch.float32), normal(T, H)
    r = d.moe_route(logits, k)
    q, xs = d.quantize_int8(X)
    wq, ws = (t.view(E, N, -1).squeeze(-1) for t in d.quantize_int8(W.view(E * N, H)))
    w2, s2 = (t.view(E, H, -1).squeeze(-1) for t in d.quantize_int8(normal(E * H, N // 2)))
    o = r.group_offsets
    return {
        "grouped_gemm_fwd": lambda s: d.grouped_gemm_fwd(X, W, o, stream=s),
        "grouped_gemm_dgrad": lambda s: d.grouped_gemm_dgrad(G, W, o, stream=s),
        "grouped_gemm_wgrad": lambda s: d.grouped_gemm_wgrad(X, G, o, stream=s),
        "batched_gemm_fwd": lambda s: d.batched_gemm_fwd(X.view(E, -1, H), W, stream=s),
        "batched_gemm_dgrad": lambda s: d.batched_gemm_dgrad(G.view(E, -1, N), W, stream=s),
        "batched_gemm_wgrad": lambda s: d.batched_gemm_wgrad(X.view(E, -1, H), G.view(E, -1, N), stream=s),
        "router_gemm_fp32_bf16x3": lambda s: d.router_gemm_fp32_bf16x3(X.float(), W[0].float(), stream=s),
        "moe_route": lambda s: d.moe_route(logits, k, stream=s),
        "moe_route_grad": lambda s: d.moe_route_grad(dw, logits, r.experts, r.weights, stream=s),
        "moe_dispatch": lambda s: d.moe_dispatch(dout, r.positions, stream=s),
        "moe_combine": lambda s: d.moe_combine(X, r.positions, r.weights, stream=s),
        "moe_combine_grad": lambda s: d.moe_combine_grad(dout, X, r.positions, r.weights, stream=s),
        "quantize_int8": lambda s: d.quantize_int8(dout, r.positions, stream=s),
        "grouped_gemm_int8": lambda s: d.grouped_gemm_int8(q, xs, wq, ws, o, stream=s),
        "gemm_int8": lambda s: d.gemm_int8(q, xs, wq[0], ws[0], stream=s),
        "moe_ffn_int8": lambda s: d.moe_ffn_int8(dout, logits, wq, ws, w2, s2, k, stream=s),
    }


@pytest.mark.parametrize("name", ["grouped_gemm_fwd", "grouped_gemm_dgrad", "grouped_gemm_wgrad", "batched_gemm_fwd",
                                  "batched_gemm_dgrad", "batched_gemm_wgrad", "router_gemm_fp32_bf16x3", "moe_route",
                                  "moe_route_grad", "moe_dispatch", "moe_combine", "moe_combine_grad", "quantize_int8",
                                  "grouped_gemm_int8", "gemm_int8", "moe_ffn_int8"])
def test_results_on_a_given_stream(drgg, name):
    call = calls(drgg)[name]
    side = torch.cuda.Stream()
    want = call(None)
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    want, got = (x if isinstance(x, tuple) else (x,) for x in (want, got))
    for a, b in zip(want, got):
        assert torch.equal(a, b)
        assert home_stream(a) == torch.cuda.current_stream().cuda_stream
        assert home_stream(b) == side.cuda_stream


@pytest.mark.parametrize("name", ["grouped_gemm_fwd", "moe_route", "moe_ffn_int8"])
def test_captured_on_a_forked_stream(drgg, name):
    """A call on a stream that a capture forks to: every replay gives the eager result."""
    call = calls(drgg)[name]
    want = call(None)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
    want, got = (x if isinstance(x, tuple) else (x,) for x in (want, got))
    for _ in range(3):
        for t in got:
            t.zero_()
        call(None)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
