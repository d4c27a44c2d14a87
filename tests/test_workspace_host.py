"""A workspace whose elements share memory reports more bytes than it has (an
expanded tensor): every call refuses it before anything is launched.  The
launches are stand-ins: runs on the CPU."""
import pytest

from tests.test_streams_host import StubLib, drgg  # noqa: F401  (the fixture that loads the library)

torch = pytest.importorskip("torch")


@pytest.fixture
def launched(drgg, monkeypatch):  # noqa: F811
    import contextlib
    seen = []

    class Lib(StubLib):
        def __getattr__(self, name):
            f = super().__getattr__(name)
            if any(q in name for q in ("size", "plan", "split", "chunking")):
                return f
            return lambda *a: seen.append(name) or 0
    monkeypatch.setattr(drgg, "lib", Lib(drgg.lib))
    monkeypatch.setattr(drgg, "_need", lambda *a: None)
    monkeypatch.setattr(drgg, "_need_rows", lambda *a: None)
    monkeypatch.setattr(drgg, "_stream", lambda *a: None)
    monkeypatch.setattr(drgg, "_RAW_STREAM", False)
    monkeypatch.setattr(drgg, "_on_one_device", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    return seen


def calls(d):
    bf, i32 = torch.bfloat16, torch.int32
    X, G, W, offsets = torch.zeros(6144, 16, dtype=bf), torch.zeros(6144, 32, dtype=bf), torch.zeros(2, 32, 16, dtype=bf), torch.zeros(3, dtype=i32)
    b = [t.view(2, 3072, -1) for t in (X, G)]
    w1, s1, w2, s2 = torch.zeros(2, 32, 16, dtype=torch.int8), torch.zeros(2, 32), torch.zeros(2, 16, 16, dtype=torch.int8), torch.zeros(2, 16)
    return {
        "grouped_gemm_dgrad": lambda w: d.grouped_gemm_dgrad(G, W, offsets, workspace=w),
        "grouped_gemm_wgrad": lambda w: d.grouped_gemm_wgrad(X, G, offsets, workspace=w),
        "batched_gemm_dgrad": lambda w: d.batched_gemm_dgrad(b[1], W, workspace=w),
        "batched_gemm_wgrad": lambda w: d.batched_gemm_wgrad(b[0], b[1], workspace=w),
        "router_gemm_fp32_bf16x3": lambda w: d.router_gemm_fp32_bf16x3(torch.zeros(300, 4096), torch.zeros(64, 4096), workspace=w),
        "moe_route": lambda w: d.moe_route(torch.zeros(130, 8), 2, workspace=w),
        "moe_ffn_int8": lambda w: d.moe_ffn_int8(X[:6], torch.zeros(6, 2), w1, s1, w2, s2, 1, workspace=w),
    }


def test_zeroed_workspace_must_be_contiguous(drgg, launched):  # noqa: F811
    with pytest.raises(ValueError, match="contiguous"):
        drgg.workspace_init(torch.zeros(1, dtype=torch.uint8).expand(1 << 20))
    assert not launched
    drgg.workspace_init(torch.zeros(64, dtype=torch.uint8))
    assert launched


@pytest.mark.parametrize("name", sorted(calls(None)))
def test_workspace_must_be_contiguous(drgg, launched, name):  # noqa: F811
    call = calls(drgg)[name]
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(1 << 30), torch.zeros((2, 64), dtype=torch.uint8)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous"):
            call(bad)
    assert not launched
    call(torch.empty(1 << 20, dtype=torch.uint8))
    assert launched
