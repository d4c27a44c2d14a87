"""Buffers whose elements or bytes pass 32 bits: the 4-bit operators, the kept
activation and the selection by scores on them, against the same calls on their
last rows alone (their results do not depend on the other rows) or against
moe_route."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def drgg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as d
    yield d
    torch.cuda.empty_cache()


def filled(shape, dtype, seed):
    """Normal values made in pieces (a random FP32 tensor of the whole size would take twice the memory)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device="cuda")
    for part in t.split(1 << 18):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return t


def test_quantize(drgg):
    T, K = (1 << 21) + 77, 2080   # 2^32.02 values
    x = filled((T, K), torch.bfloat16, 0)
    q, s = drgg.quantize_mxfp4(x)
    part = x[-300:].contiguous()
    qp, sp = drgg.quantize_mxfp4(part)
    assert torch.equal(q[-300:], qp) and torch.equal(s[:, -300:], sp)
    del x
    assert torch.equal(drgg.dequantize_mxfp4(q, s)[-300:], drgg.dequantize_mxfp4(qp, sp))


@pytest.mark.parametrize("gated", [False, True])
def test_product_of_many_rows(drgg, gated):
    M, N, K = (1 << 21) + 77, 2080, 4128   # 4.3 GB of codes, 2^32.02 results
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(125, 130, (17, M, 8), generator=g, device="cuda", dtype=torch.uint8)
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(125, 130, (17, N, 8), generator=g, device="cuda", dtype=torch.uint8)
    y = drgg.gemm_mxfp4(q, s, w, ws, gated=gated)
    at = slice(M - 2000, M)   # sums that fit 24 bits: the same in every program
    assert torch.equal(y[at], drgg.gemm_mxfp4(q[at].contiguous(), s[:, at].contiguous(), w, ws, gated=gated))


def test_product_of_many_weights(drgg):
    E, N, K = 520, 4096, 4160   # 4.4 GB of codes
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(125, 130, (17, E, N, 8), generator=g, device="cuda", dtype=torch.uint8)
    for rows in (2, 70):   # the few-row blocks and the tiles
        M = E * rows
        q = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = torch.randint(125, 130, (17, M, 8), generator=g, device="cuda", dtype=torch.uint8)
        offsets = torch.arange(E + 1, device="cuda", dtype=torch.int32) * rows
        y = drgg.grouped_gemm_mxfp4(q, s, w, ws, offsets, out_dtype=torch.float32)
        for e in (E // 2, E - 1):
            at = slice(e * rows, e * rows + rows)
            assert torch.equal(y[at], drgg.gemm_mxfp4(q[at].contiguous(), s[:, at].contiguous(), w[e],
                                                      ws[:, e].contiguous(), out_dtype=torch.float32))


def test_gate(drgg):
    T, I = (1 << 20) + 5, 2056   # 2^32.02 values in GU
    GU = filled((T, 2 * I), torch.bfloat16, 3)
    positions = torch.arange(T, device="cuda", dtype=torch.int32).view(T, 1)
    weights = torch.rand(T, 1, device="cuda")
    h, q, s = drgg.moe_gate_int8(GU, positions, weights)
    n = 200
    at = positions[:n].contiguous()
    last = drgg.moe_gate_int8(GU[-n:].contiguous(), at, weights[-n:].contiguous())
    for a, b in zip((h, q, s), last):
        assert torch.equal(a[-n:], b)
    del GU
    grads = drgg.moe_gate_int8_grad(h, q, s, positions, weights)
    part = drgg.moe_gate_int8_grad(last[0], last[1], last[2], at, weights[-n:].contiguous())
    for a, b in zip(grads, part):
        assert torch.equal(a[-n:], b)


def test_scores(drgg):
    T, E, k = (1 << 22) + 9, 520, 2   # 2^31.02 logits
    x = filled((T, E), torch.float32, 4)
    want, got = drgg.moe_route(x, k), drgg.moe_route_scores(x, k, drgg.Scoring("softmax"))
    for name in ("experts", "positions", "group_offsets", "tokens"):
        assert torch.equal(getattr(want, name), getattr(got, name))
    sc = drgg.Scoring(bias=torch.linspace(-0.5, 0.5, E, device="cuda"))
    r = drgg.moe_route_scores(x, k, sc)
    n = 500
    part = drgg.moe_route_scores(x[-n:].contiguous(), k, sc)
    assert torch.equal(r.experts[-n:], part.experts) and torch.equal(r.weights[-n:], part.weights)
    dw = torch.randn(T, k, device="cuda")
    del want, got
    d = drgg.moe_route_scores_grad(dw, x, r.experts, r.weights, sc)
    assert torch.equal(d[-n:], drgg.moe_route_scores_grad(dw[-n:].contiguous(), x[-n:].contiguous(), part.experts,
                                                          part.weights, sc))
