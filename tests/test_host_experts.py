"""Host-side tests of the scored selection, the 4-bit products and the kept
activation (no GPU needed): argument checks reject bad calls before anything
reaches the GPU, and the workspace sizes."""
import ctypes
import os
import shutil
import subprocess

import pytest

from tests.test_host import A16, drgg  # noqa: F401  (the fixture that loads the library)
from tests.test_sanitize import HERE, ROCM, ROOT, SAN, _run

OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE = 0, 1, 2, 3, 5


def scoring(drgg, score=1, groups=4, top_groups=2, best=2, renormalize=1, scale=2.5, bias=A16):  # noqa: F811
    return drgg.ScoringStruct(score, groups, top_groups, best, renormalize, scale, bias)


BAD_SCORING = (dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=65), dict(top_groups=0),
               dict(top_groups=5), dict(best=0), dict(best=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(top_groups=1, groups=8))   # one expert, k = 2


def test_route_scores_argument_checks(drgg):  # noqa: F811
    def route(c=None, logits=A16, T=100, E=8, k=2, experts=A16, weights=A16, offsets=A16, positions=A16, tokens=0, ws=A16,
              ws_bytes=1 << 20, none=False):
        return drgg.lib.moe_route_scores(logits, T, E, k, None if none else c or scoring(drgg), experts, weights, offsets,
                                         positions, tokens, ws, ws_bytes, None)

    assert route(none=True) == EINVAL
    for bad in BAD_SCORING:
        assert route(scoring(drgg, **bad)) == EINVAL, bad
    assert route(scoring(drgg, bias=A16 + 2)) == EALIGN
    for bad in (dict(E=0), dict(E=1028), dict(k=0), dict(k=9), dict(E=1024, k=65), dict(logits=0), dict(experts=0),
                dict(weights=0), dict(offsets=0), dict(positions=0)):
        assert route(**bad) == EINVAL, bad
    for bad in (dict(T=-1), dict(T=2 ** 27 + 1), dict(T=2 ** 26, E=64, k=32)):
        assert route(**bad) == ESHAPE, bad
    for bad in (dict(logits=A16 + 4), dict(experts=A16 + 2), dict(weights=A16 + 1), dict(offsets=A16 + 2),
                dict(positions=A16 + 2), dict(tokens=A16 + 2), dict(ws=A16 + 8)):
        assert route(**bad) == EALIGN, bad
    need = drgg.route_workspace_size(100, 8, 2)
    for bad in (dict(ws=0), dict(ws_bytes=need - 1)):
        assert route(**bad) == EWORKSPACE, bad


def test_route_scores_grad_argument_checks(drgg):  # noqa: F811
    def grad(c=None, dw=A16, logits=A16, experts=A16, weights=A16, T=4, E=8, k=2, out=A16):
        return drgg.lib.moe_route_scores_grad(dw, logits, experts, weights, T, E, k, c or scoring(drgg), out, None)

    assert drgg.lib.moe_route_scores_grad(A16, A16, A16, A16, 4, 8, 2, None, A16, None) == EINVAL
    for bad in (dict(score=2), dict(scale=0.0), dict(scale=float("nan"))):
        assert grad(scoring(drgg, **bad)) == EINVAL, bad
    for bad, want in ((dict(dw=0), EINVAL), (dict(logits=0), EINVAL), (dict(experts=0), EINVAL), (dict(weights=0), EINVAL),
                      (dict(out=0), EINVAL), (dict(k=9), EINVAL), (dict(T=-1), ESHAPE), (dict(out=A16 + 8), EALIGN),
                      (dict(logits=A16 + 8), EALIGN), (dict(dw=A16 + 2), EALIGN)):
        assert grad(**bad) == want, bad
    assert grad(T=0, dw=0, logits=0, experts=0, weights=0, out=0) == OK


def test_mxfp4_row_argument_checks(drgg):  # noqa: F811
    def quantize(X=A16, dt=0, T=4, K=64, q=A16, s=A16):
        return drgg.lib.quantize_mxfp4(X, dt, T, K, q, s, None)

    def dequantize(X=A16, dt=0, T=4, K=64, q=A16, s=A16):
        return drgg.lib.dequantize_mxfp4(q, s, T, K, dt, X, None)

    for call in (quantize, dequantize):
        for bad, want in ((dict(X=0), EINVAL), (dict(q=0), EINVAL), (dict(s=0), EINVAL), (dict(dt=2), EINVAL),
                          (dict(T=-1), ESHAPE), (dict(T=2 ** 31), ESHAPE), (dict(K=0), ESHAPE), (dict(K=2 ** 22 + 32), ESHAPE),
                          (dict(K=80), EALIGN), (dict(X=A16 + 8), EALIGN), (dict(q=A16 + 8), EALIGN), (dict(s=A16 + 4), EALIGN)):
            assert call(**bad) == want, (call, bad)
        assert call(T=0, X=0, q=0, s=0) == OK


def test_mxfp4_product_argument_checks(drgg):  # noqa: F811
    def grouped(X=A16, xs=A16, W=A16, ws=A16, offs=A16, rows=0, T=0, E=2, M=8, N=64, K=64, gated=0, dt=0, Y=A16):
        return drgg.lib.grouped_gemm_mxfp4(X, xs, W, ws, offs, rows, T, E, M, N, K, gated, dt, Y, None)

    def dense(X=A16, xs=A16, W=A16, ws=A16, M=8, N=64, K=64, gated=0, dt=0, Y=A16):
        return drgg.lib.gemm_mxfp4(X, xs, W, ws, M, N, K, gated, dt, Y, None)

    both = ((dict(X=0), EINVAL), (dict(xs=0), EINVAL), (dict(W=0), EINVAL), (dict(ws=0), EINVAL), (dict(Y=0), EINVAL),
            (dict(dt=2), EINVAL), (dict(M=-1), ESHAPE), (dict(M=2 ** 31), ESHAPE), (dict(N=0), ESHAPE),
            (dict(N=2 ** 22 + 8), ESHAPE), (dict(K=0), ESHAPE), (dict(K=2 ** 22 + 32), ESHAPE), (dict(N=12), EALIGN),
            (dict(N=24, gated=1), EALIGN), (dict(N=8, gated=1), ESHAPE), (dict(K=48), EALIGN), (dict(X=A16 + 8), EALIGN),
            (dict(W=A16 + 8), EALIGN), (dict(Y=A16 + 8), EALIGN), (dict(ws=A16 + 4), EALIGN), (dict(xs=A16 + 4), EALIGN))
    for bad, want in both:
        assert grouped(**bad) == want, bad
        assert dense(**bad) == want, bad
    for bad, want in ((dict(offs=0), EINVAL), (dict(E=0), EINVAL), (dict(E=1025), EINVAL), (dict(offs=A16 + 2), EALIGN),
                      (dict(rows=A16, T=0), ESHAPE), (dict(rows=A16, T=2 ** 31 // 32), ESHAPE),
                      (dict(rows=A16 + 2, T=8), EALIGN)):
        assert grouped(**bad) == want, bad
    assert grouped(M=0, X=0, xs=0, Y=0) == OK and dense(M=0, X=0, xs=0, Y=0) == OK


def test_mxfp4_ffn_argument_checks(drgg):  # noqa: F811
    def ffn(X=A16, logits=A16, w1=A16, s1=A16, w2=A16, s2=A16, T=4, E=8, k=2, H=64, inner=32, c=None, out=A16, ws=A16,
            ws_bytes=1 << 30):
        return drgg.lib.moe_ffn_mxfp4(X, logits, w1, s1, w2, s2, T, E, k, H, inner, c, out, ws, ws_bytes, None)

    need = drgg.ffn_mxfp4_workspace_size(4, 8, 2, 64, 32)
    for bad, want in ((dict(X=0), EINVAL), (dict(logits=0), EINVAL), (dict(w1=0), EINVAL), (dict(s1=0), EINVAL),
                      (dict(w2=0), EINVAL), (dict(s2=0), EINVAL), (dict(out=0), EINVAL), (dict(k=9), EINVAL),
                      (dict(E=0), EINVAL), (dict(T=-1), ESHAPE), (dict(H=0), ESHAPE), (dict(inner=16), ESHAPE),
                      (dict(H=2 ** 22 + 32), ESHAPE), (dict(inner=2 ** 21 + 32), ESHAPE), (dict(T=2 ** 27, H=64), ESHAPE),
                      (dict(H=80), EALIGN), (dict(inner=48), EALIGN), (dict(X=A16 + 8), EALIGN), (dict(s1=A16 + 4), EALIGN),
                      (dict(out=A16 + 8), EALIGN), (dict(ws=0), EWORKSPACE), (dict(ws_bytes=need - 1), EWORKSPACE),
                      (dict(ws=A16 + 8), EALIGN), (dict(c=scoring(drgg, best=3)), EINVAL),
                      (dict(c=scoring(drgg, bias=A16 + 2)), EALIGN)):
        assert ffn(**bad) == want, bad
    assert ffn(T=0, X=0, logits=0, out=0, ws=0, ws_bytes=0) == OK
    size = ctypes.c_size_t()
    assert drgg.lib.moe_ffn_mxfp4_workspace_size(4, 8, 2, 64, 32, None) == EINVAL
    assert drgg.lib.moe_ffn_mxfp4_workspace_size(2 ** 27, 8, 2, 64, 32, ctypes.byref(size)) == ESHAPE


def test_gate_argument_checks(drgg):  # noqa: F811
    def forward(GU=A16, pos=A16, w=A16, T=4, k=2, inner=64, h=A16, q=A16, s=A16):
        return drgg.lib.moe_gate_int8(GU, pos, w, T, k, inner, h, q, s, None)

    def grad(dh=A16, q=A16, s=A16, pos=A16, w=A16, T=4, k=2, inner=64, dGU=A16, h=A16, dw=A16):
        return drgg.lib.moe_gate_int8_grad(dh, q, s, pos, w, T, k, inner, dGU, h, dw, None)

    for call in (forward, grad):
        for bad, want in ((dict(pos=0), EINVAL), (dict(w=0), EINVAL), (dict(h=0), EINVAL), (dict(q=0), EINVAL),
                          (dict(s=0), EINVAL), (dict(k=0), EINVAL), (dict(k=65), EINVAL), (dict(T=-1), ESHAPE),
                          (dict(T=2 ** 30, k=2), ESHAPE), (dict(inner=0), ESHAPE), (dict(inner=2 ** 21 + 8), ESHAPE),
                          (dict(inner=20), EALIGN), (dict(h=A16 + 8), EALIGN), (dict(q=A16 + 4), EALIGN),
                          (dict(s=A16 + 2), EALIGN), (dict(pos=A16 + 2), EALIGN)):
            assert call(**bad) == want, (call, bad)
    assert forward(GU=0) == EINVAL and forward(GU=A16 + 8) == EALIGN
    assert grad(dh=0) == EINVAL and grad(dGU=A16 + 8) == EALIGN and grad(dw=0) == EINVAL and grad(dw=A16 + 2) == EALIGN
    assert forward(T=0, GU=0, pos=0, w=0, h=0, q=0, s=0) == OK
    assert grad(T=0, dh=0, q=0, s=0, pos=0, w=0, dGU=0, h=0, dw=0) == OK


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="needs g++ and the HIP headers")
def test_host_code_under_sanitizers(tmp_path):
    """api_experts.cpp with stubs for the launchers, which check the serving block's workspace layout."""
    exe = str(tmp_path / "experts_driver")
    csrc = os.path.join(ROOT, "dense_ragged_grouped_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
                    "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(HERE, "experts_driver.cpp"), os.path.join(csrc, "api_experts.cpp"), "-o", exe], check=True)
    _run(exe, tmp_path)
