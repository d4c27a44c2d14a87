"""Where the results of a call with stream= come from: memory of the stream
that writes them (what is free on the caller's stream may still be in use
there), marked as used by the caller's stream too (so that it is not handed
out again on the writing one while the caller reads it).  The launches, the
streams and the allocations' streams are stand-ins: runs on the CPU."""
import contextlib

import pytest

from tests.test_host import drgg  # noqa: F401  (the fixture that loads the library)

torch = pytest.importorskip("torch")

HOST_QUERIES = ("size", "plan", "split", "chunking")


class StubLib:
    """Host queries reach the library; everything that launches does nothing."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        if any(q in name for q in HOST_QUERIES):
            return getattr(self.lib, name)
        return lambda *args: 0


@pytest.fixture
def world(drgg, monkeypatch):  # noqa: F811
    home, side = object(), object()
    now = [home]
    born, shared = {}, {}

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    new_empty, empty = torch.Tensor.new_empty, torch.empty

    def note(t):
        born[t.untyped_storage()._cdata] = now[-1]
        return t
    monkeypatch.setattr(torch.Tensor, "new_empty", lambda self, *a, **k: note(new_empty(self, *a, **k)))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: note(empty(*a, **k)))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda self, s: shared.setdefault(self.untyped_storage()._cdata, set()).add(s))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(drgg, "lib", StubLib(drgg.lib))
    monkeypatch.setattr(drgg, "_need", lambda *a: None)
    monkeypatch.setattr(drgg, "_need_rows", lambda *a: None)
    monkeypatch.setattr(drgg, "_stream", lambda *a: None)
    monkeypatch.setattr(drgg, "_workspace", lambda *a, **k: (None, 0))
    monkeypatch.setattr(drgg, "_on_one_device", lambda *a: contextlib.nullcontext())
    return home, side, born, shared


def calls(d):
    bf, i32 = torch.bfloat16, torch.int32
    X, G, W = torch.zeros(6, 16, dtype=bf), torch.zeros(6, 32, dtype=bf), torch.zeros(2, 32, 16, dtype=bf)
    offsets = torch.zeros(3, dtype=i32)
    b = [t.view(2, 3, -1) for t in (X, G)]
    logits = torch.zeros(130, 8)
    experts, weights = torch.zeros(130, 2, dtype=i32), torch.zeros(130, 2)
    positions, pw, rows = torch.zeros(6, 2, dtype=i32), torch.zeros(6, 2), torch.zeros(12, 16, dtype=bf)
    q, xs, wq, ws = torch.zeros(6, 16, dtype=torch.int8), torch.zeros(6), torch.zeros(2, 32, 16, dtype=torch.int8), torch.zeros(2, 32)
    w2, s2 = torch.zeros(2, 16, 16, dtype=torch.int8), torch.zeros(2, 16)
    return {
        "grouped_gemm_fwd": lambda s: d.grouped_gemm_fwd(X, W, offsets, stream=s),
        "grouped_gemm_dgrad": lambda s: d.grouped_gemm_dgrad(G, W, offsets, stream=s),
        "grouped_gemm_wgrad": lambda s: d.grouped_gemm_wgrad(X, G, offsets, stream=s),
        "batched_gemm_fwd": lambda s: d.batched_gemm_fwd(b[0], W, stream=s),
        "batched_gemm_dgrad": lambda s: d.batched_gemm_dgrad(b[1], W, stream=s),
        "batched_gemm_wgrad": lambda s: d.batched_gemm_wgrad(b[0], b[1], stream=s),
        "router_gemm_fp32_bf16x3": lambda s: d.router_gemm_fp32_bf16x3(torch.zeros(8, 32), torch.zeros(8, 32), stream=s),
        "moe_route": lambda s: d.moe_route(logits, 2, stream=s),
        "moe_route_grad": lambda s: d.moe_route_grad(weights, logits, experts, weights, stream=s),
        "moe_dispatch": lambda s: d.moe_dispatch(X, positions, stream=s),
        "moe_combine": lambda s: d.moe_combine(rows, positions, pw, stream=s),
        "moe_combine_grad": lambda s: d.moe_combine_grad(X, rows, positions, pw, stream=s),
        "quantize_int8": lambda s: d.quantize_int8(X, stream=s),
        "quantize_int8_grouped": lambda s: d.quantize_int8(X, positions, stream=s),
        "grouped_gemm_int8": lambda s: d.grouped_gemm_int8(q, xs, wq, ws, offsets, stream=s),
        "gemm_int8": lambda s: d.gemm_int8(q, xs, wq[0], ws[0], stream=s),
        "moe_ffn_int8": lambda s: d.moe_ffn_int8(X, torch.zeros(6, 2), wq, ws, w2, s2, 1, stream=s),
    }


@pytest.mark.parametrize("name", sorted(calls(None)))
def test_results_on_a_given_stream(drgg, world, name):  # noqa: F811
    home, side, born, shared = world
    got = calls(drgg)[name](side)
    for t in got if isinstance(got, tuple) else (got,):
        at = t.untyped_storage()._cdata
        assert born[at] is side
        assert shared.get(at) == {home}


def test_the_given_stream_is_the_current_one(drgg, world):  # noqa: F811
    """Nothing to record then."""
    home, _, born, shared = world
    got = calls(drgg)["moe_combine"](home)
    assert born[got.untyped_storage()._cdata] is home and not shared


@pytest.mark.parametrize("name", sorted(calls(None)))
def test_results_on_the_current_stream(drgg, world, name, monkeypatch):  # noqa: F811
    home, _, born, shared = world
    monkeypatch.setattr(drgg, "_RAW_STREAM", False)   # the accessors of the current stream's handle need a GPU
    got = calls(drgg)[name](None)
    for t in got if isinstance(got, tuple) else (got,):
        assert born[t.untyped_storage()._cdata] is home
    assert not shared
