"""Calls with stream= of the selection by scores, the 4-bit operators and the
kept activation: where their results come from, on the CPU with stand-ins
(tests/test_streams_host.py) and on the GPU (tests/test_gpu_streams.py)."""
import pytest

from tests.test_host import drgg  # noqa: F401  (the fixture that loads the library)
from tests.test_streams_host import world  # noqa: F401

torch = pytest.importorskip("torch")


def calls(d, device="cpu"):
    def of(*shape, dtype=torch.bfloat16):
        return torch.ones(*shape, dtype=dtype, device=device)
    u8, f32 = torch.uint8, torch.float32
    X, logits, dw = of(130, 64), of(130, 4, dtype=f32), of(130, 2, dtype=f32)
    experts = torch.arange(2, dtype=torch.int32, device=device).repeat(130, 1)
    positions = torch.arange(260, dtype=torch.int32, device=device).view(130, 2)
    GU, dh, kept, scale = of(260, 128), of(260, 64), of(260, 128, dtype=torch.int8), of(260, 2, dtype=f32)
    q, s = of(130, 32, dtype=u8), of(1, 130, 8, dtype=u8)
    w1, s1, w2, s2 = of(4, 64, 32, dtype=u8), of(1, 4, 64, 8, dtype=u8), of(4, 64, 16, dtype=u8), of(1, 4, 64, 8, dtype=u8)
    offsets = torch.tensor([0, 30, 30, 100, 130], dtype=torch.int32, device=device)
    return {
        "moe_route_scores": lambda st: d.moe_route_scores(logits, 2, stream=st),
        "moe_route_scores_grad": lambda st: d.moe_route_scores_grad(dw, logits, experts, dw, stream=st),
        "quantize_mxfp4": lambda st: d.quantize_mxfp4(X, stream=st),
        "dequantize_mxfp4": lambda st: d.dequantize_mxfp4(q, s, stream=st),
        "grouped_gemm_mxfp4": lambda st: d.grouped_gemm_mxfp4(q, s, w1, s1, offsets, stream=st),
        "gemm_mxfp4": lambda st: d.gemm_mxfp4(q, s, w1[0], s1[:, 0].contiguous(), stream=st),
        "moe_ffn_mxfp4": lambda st: d.moe_ffn_mxfp4(X, logits, w1, s1, w2, s2, 2, scoring=d.Scoring(), stream=st),
        "moe_gate_int8": lambda st: d.moe_gate_int8(GU, positions, dw, stream=st),
        "moe_gate_int8_grad": lambda st: d.moe_gate_int8_grad(dh, kept, scale, positions, dw, stream=st),
    }


NAMES = ["moe_route_scores", "moe_route_scores_grad", "quantize_mxfp4", "dequantize_mxfp4", "grouped_gemm_mxfp4", "gemm_mxfp4",
         "moe_ffn_mxfp4", "moe_gate_int8", "moe_gate_int8_grad"]


def several(x):
    return x if isinstance(x, tuple) else (x,)


@pytest.mark.parametrize("name", NAMES)
def test_results_on_a_given_stream(drgg, world, name):  # noqa: F811
    home, side, born, shared = world
    for t in several(calls(drgg)[name](side)):
        at = t.untyped_storage()._cdata
        assert born[at] is side
        assert shared.get(at) == {home}


@pytest.mark.parametrize("name", NAMES)
def test_results_on_the_current_stream(drgg, world, name, monkeypatch):  # noqa: F811
    home, _, born, shared = world
    monkeypatch.setattr(drgg, "_RAW_STREAM", False)   # the accessors of the current stream's handle need a GPU
    for t in several(calls(drgg)[name](None)):
        assert born[t.untyped_storage()._cdata] is home
    assert not shared


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_on_the_gpu(name):
    """On a given stream and captured on a forked one: the eager result, in the given stream's memory."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as d
    from tests.test_gpu_streams import home_stream
    call = calls(d, "cuda")[name]
    want = several(call(None))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = several(call(side))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b) and home_stream(b) == side.cuda_stream
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = several(call(side))
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in got:
            t.zero_()
        call(None)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
