"""Logits and their gradient need 16-byte alignment only where the kernels move
four at a time, for E a multiple of 4; with another E a slice of a batch's
tokens starts anywhere."""
import pytest

from tests.test_host import A16, drgg  # noqa: F401  (the fixture that loads the library)

OK, EALIGN, EWORKSPACE = 0, 3, 5


@pytest.mark.parametrize("E,step,want", [(9, 4, True), (57, 12, True), (1023, 8, True), (9, 2, False), (8, 4, False),
                                         (1024, 8, False), (8, 16, True)])
def test_alignment_checks(drgg, E, step, want):  # noqa: F811
    """Nothing is launched: the workspace is missing, or there are no tokens."""
    at = A16 + step
    got = drgg.lib.moe_route(at, 100, E, 1, 1, A16, A16, A16, A16, 0, 0, 0, None)
    assert got == (EWORKSPACE if want else EALIGN)
    got = drgg.lib.moe_ffn_int8(A16, at, A16, A16, A16, A16, 100, E, 1, 64, 32, 1, A16, 0, 0, None)
    assert got == (EWORKSPACE if want else EALIGN)
    for logits, dlogits in ((at, A16), (A16, at)):
        got = drgg.lib.moe_route_grad(A16, logits, A16, A16, 0, E, 1, 1, dlogits, None)
        assert got == (OK if want else EALIGN)


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(57, 4), (9, 2), (1022, 8)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_slices_of_logits(drgg, E, k, renormalize):  # noqa: F811
    """A slice of the tokens gives the bits of its copy, forward and gradient; nothing beside it is written."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    T = 131
    whole = torch.randn((T + 2, E), generator=g, device="cuda")
    dw = torch.randn((T, k), generator=g, device="cuda")
    part, copy = whole[1:T + 1], whole[1:T + 1].clone()
    assert part.data_ptr() % 16
    r, want = drgg.moe_route(part, k, renormalize=renormalize), drgg.moe_route(copy, k, renormalize=renormalize)
    for a, b in zip(r, want):
        assert torch.equal(a, b)
    out = torch.full((T + 2, E), 7.0, device="cuda")
    drgg.moe_route_grad(dw, part, r.experts, r.weights, renormalize=renormalize, out=out[1:T + 1])
    assert torch.equal(out[1:T + 1], drgg.moe_route_grad(dw, copy, r.experts, r.weights, renormalize=renormalize))
    assert bool((out[0] == 7).all()) and bool((out[T + 1] == 7).all())
