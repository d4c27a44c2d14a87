"""Host-side tests of the expert-layer entry points (no GPU needed): argument
checks reject bad calls before anything reaches the GPU, and the workspace
sizes."""
import pytest

from tests.test_host import A16, drgg  # noqa: F401  (the fixture that loads the library)

OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE = 0, 1, 2, 3, 5


def route(drgg, logits=A16, T=100, E=8, k=2, experts=A16, weights=A16, offsets=A16, positions=A16, tokens=0, ws=A16,
          ws_bytes=1 << 20):
    return drgg.lib.moe_route(logits, T, E, k, 1, experts, weights, offsets, positions, tokens, ws, ws_bytes, None)


def test_route_argument_checks(drgg):  # noqa: F811
    for bad in (dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=100, k=65), dict(logits=0), dict(experts=0),
                dict(weights=0), dict(offsets=0), dict(positions=0)):
        assert route(drgg, **bad) == EINVAL, bad
    for bad in (dict(T=-1), dict(T=2 ** 27 + 1), dict(T=2 ** 26, E=64, k=32)):
        assert route(drgg, **bad) == ESHAPE, bad
    for bad in (dict(logits=A16 + 4), dict(experts=A16 + 2), dict(weights=A16 + 1), dict(offsets=A16 + 2),
                dict(positions=A16 + 2), dict(tokens=A16 + 2), dict(ws=A16 + 8)):
        assert route(drgg, **bad) == EALIGN, bad
    need = drgg.route_workspace_size(100, 8, 2)
    assert need > 0
    for bad in (dict(ws=0), dict(ws_bytes=need - 1)):
        assert route(drgg, **bad) == EWORKSPACE, bad
    grad = drgg.lib.moe_route_grad
    assert grad(0, A16, A16, A16, 4, 8, 2, 1, A16, None) == EINVAL
    assert grad(A16, A16, A16, A16, 4, 8, 9, 1, A16, None) == EINVAL
    assert grad(A16, A16, A16, A16, 4, 8, 2, 1, A16 + 8, None) == EALIGN
    assert grad(0, 0, 0, 0, 0, 8, 2, 1, 0, None) == OK        # no tokens: nothing to do


def test_route_workspace(drgg):  # noqa: F811
    size = drgg.route_workspace_size
    assert size(0, 8, 2) == size(64, 8, 2) == 0
    assert size(65, 8, 2) == 2 * 8 and size(65, 9, 2) == 2 * 12          # bytes, experts rounded up to four
    assert size(64 * 512, 256, 8) == 512 * 256
    assert size(64 * 512 + 1, 256, 8) == 514 * 256 * 4                   # words and the totals
    assert size(2 ** 27, 1024, 8) == (2 ** 21 + 1) * 1024 * 4
    for bad in ((-1, 8, 2), (10, 0, 1), (10, 8, 9)):
        with pytest.raises(drgg.DrggError):
            size(*bad)


def test_row_argument_checks(drgg):  # noqa: F811
    lib = drgg.lib

    def dispatch(X=A16, pos=A16, T=4, k=2, H=64, dt=0, rows=A16):
        return lib.moe_dispatch(X, pos, T, k, H, dt, rows, None)

    def combine(rows=A16, pos=A16, w=A16, T=4, k=2, H=64, dt=0, out=A16):
        return lib.moe_combine(rows, pos, w, T, k, H, dt, out, None)

    def grad(dout=A16, rows=A16, pos=A16, w=A16, T=4, k=2, H=64, dt=0, drows=A16, dw=A16):
        return lib.moe_combine_grad(dout, rows, pos, w, T, k, H, dt, drows, dw, None)

    for call in (dispatch, combine, grad):
        for bad, want in ((dict(pos=0), EINVAL), (dict(rows=0), EINVAL), (dict(dt=2), EINVAL), (dict(k=0), EINVAL),
                          (dict(k=65), EINVAL), (dict(T=-1), ESHAPE), (dict(T=2 ** 31), ESHAPE),
                          (dict(T=2 ** 30, k=2), ESHAPE), (dict(H=0), ESHAPE), (dict(H=2 ** 22 + 8), ESHAPE),
                          (dict(H=20), EALIGN), (dict(rows=A16 + 8), EALIGN), (dict(pos=A16 + 2), EALIGN)):
            assert call(**bad) == want, (call, bad)
        assert call(T=0) == OK
    assert grad(w=0) == EINVAL and grad(dw=A16 + 2) == EALIGN and grad(drows=A16 + 4) == EALIGN
    assert combine(w=A16 + 2) == EALIGN and combine(out=0) == EINVAL and dispatch(X=A16 + 8) == EALIGN


def test_quantize_argument_checks(drgg):  # noqa: F811
    def quantize(X=A16, dt=0, T=4, K=64, pos=0, k=1, q=A16, scale=A16):
        return drgg.lib.quantize_int8(X, dt, T, K, pos, k, q, scale, None)

    for bad, want in ((dict(X=0), EINVAL), (dict(q=0), EINVAL), (dict(scale=0), EINVAL), (dict(dt=2), EINVAL),
                      (dict(k=2), EINVAL), (dict(T=-1), ESHAPE), (dict(K=0), ESHAPE), (dict(K=2 ** 22 + 16), ESHAPE),
                      (dict(K=72), EALIGN), (dict(X=A16 + 8), EALIGN), (dict(q=A16 + 8), EALIGN),
                      (dict(pos=A16 + 1, k=2), EALIGN), (dict(scale=A16 + 2), EALIGN)):
        assert quantize(**bad) == want, bad
    assert quantize(T=0) == OK and quantize(T=0, k=2) == OK


def test_int8_argument_checks(drgg):  # noqa: F811
    def grouped(X=A16, xs=A16, W=A16, ws=A16, offs=A16, rows=0, T=0, E=2, M=8, N=64, K=64, gated=0, dt=0, Y=A16):
        return drgg.lib.grouped_gemm_int8(X, xs, W, ws, offs, rows, T, E, M, N, K, gated, dt, Y, None)

    def dense(X=A16, xs=A16, W=A16, ws=A16, M=8, N=64, K=64, gated=0, dt=0, Y=A16):
        return drgg.lib.gemm_int8(X, xs, W, ws, M, N, K, gated, dt, Y, None)

    both = ((dict(X=0), EINVAL), (dict(xs=0), EINVAL), (dict(W=0), EINVAL), (dict(ws=0), EINVAL), (dict(Y=0), EINVAL),
            (dict(dt=2), EINVAL), (dict(M=-1), ESHAPE), (dict(M=2 ** 31), ESHAPE), (dict(N=0), ESHAPE),
            (dict(N=2 ** 22 + 8), ESHAPE), (dict(K=0), ESHAPE), (dict(K=131072), ESHAPE), (dict(N=12), EALIGN),
            (dict(N=24, gated=1), EALIGN), (dict(N=8, gated=1), ESHAPE), (dict(K=24), EALIGN), (dict(X=A16 + 8), EALIGN),
            (dict(W=A16 + 8), EALIGN), (dict(Y=A16 + 8), EALIGN), (dict(ws=A16 + 4), EALIGN), (dict(xs=A16 + 2), EALIGN))
    for bad, want in both:
        assert grouped(**bad) == want, bad
        assert dense(**bad) == want, bad
    for bad, want in ((dict(offs=0), EINVAL), (dict(E=0), EINVAL), (dict(E=1025), EINVAL), (dict(offs=A16 + 2), EALIGN),
                      (dict(rows=A16, T=0), ESHAPE), (dict(rows=A16, T=2 ** 31 // 64), ESHAPE),
                      (dict(rows=A16 + 2, T=8), EALIGN)):
        assert grouped(**bad) == want, bad
    assert grouped(M=0, X=0, xs=0, Y=0) == OK and dense(M=0, X=0, xs=0, Y=0) == OK


def test_ffn_argument_checks(drgg):  # noqa: F811
    def ffn(X=A16, logits=A16, w1=A16, s1=A16, w2=A16, s2=A16, T=4, E=8, k=2, H=64, inner=32, out=A16, ws=A16,
            ws_bytes=1 << 30):
        return drgg.lib.moe_ffn_int8(X, logits, w1, s1, w2, s2, T, E, k, H, inner, 1, out, ws, ws_bytes, None)

    need = drgg.ffn_workspace_size(4, 8, 2, 64, 32)
    for bad, want in ((dict(X=0), EINVAL), (dict(logits=0), EINVAL), (dict(w1=0), EINVAL), (dict(s1=0), EINVAL),
                      (dict(w2=0), EINVAL), (dict(s2=0), EINVAL), (dict(out=0), EINVAL), (dict(k=9), EINVAL),
                      (dict(E=0), EINVAL), (dict(T=-1), ESHAPE), (dict(H=0), ESHAPE), (dict(inner=8), ESHAPE),
                      (dict(H=131072), ESHAPE), (dict(H=72), EALIGN), (dict(inner=24), EALIGN), (dict(X=A16 + 8), EALIGN),
                      (dict(out=A16 + 8), EALIGN), (dict(ws=0), EWORKSPACE), (dict(ws_bytes=need - 1), EWORKSPACE),
                      (dict(ws=A16 + 8), EALIGN)):
        assert ffn(**bad) == want, bad
    assert ffn(T=0, X=0, logits=0, out=0, ws=0, ws_bytes=0) == OK
