"""Every program of the 4-bit product against exact products in 64 bits: the
few-row programs' blocks of 16, 32 and 64 tokens and their K split, and the
tiles; with and without gathered rows and the gate, BF16, FP32 and, through the
serving block, codes.

On the CPU: the shapes below run in the programs they are listed for, by the
launcher's own rule, and together reach every one.

Tolerances as in tests/test_gpu_mxfp4.py: the sums fit 24 bits and are exact.
"""
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests.test_sanitize import HERE, ROOT, SAN

T256, T128, T128x256 = 1, 2, 4
MIXED = [0, 1, 16, 17, 32, 33, 15, 2, 31, 48]

# (program, gated or None for both, counts, N, K); program: (tile, nb, waves, tok)
SHAPES = [
    ((0, 4, 4, 32), None, [0, 3, 16, 17, 33, 0, 1, 2] * 8, 528, 224),
    ((0, 4, 4, 32), None, [0, 0, 30, 1] * 16, 560, 32),
    ((0, 4, 4, 32), None, [9, 0, 20, 1] * 16, 528, 1312),
    ((0, 4, 8, 64), None, [64, 33, 17, 16, 1, 0, 130, 48, 63, 20], 1040, 352),
    ((0, 4, 8, 64), None, [700], 1040, 4128),
    ((0, 2, 8, 64), None, [64, 33, 17, 16, 1, 0, 130], 1040, 576),
    ((0, 2, 8, 64), True, [65, 33, 16], 1040, 3104),
    ((0, 1, 8, 64), False, [65, 33, 16], 1040, 3104),
    ((0, 1, 8, 64), False, [1], 4096, 2080),
    ((0, 4, 4, 64), None, [64, 33, 17, 16, 1, 0, 62, 48, 63, 20, 130, 5, 31, 32, 49, 18, 40, 7, 65, 44], 1040, 256),
    ((T128, 0, 0, 0), None, [60] * 40, 1040, 352),
    ((T256, 0, 0, 0), False, [300, 1, 4000, 257, 0, 6000], 2064, 1056),
    ((T256, 0, 0, 0), True, [300, 1, 4000, 257, 0, 6000], 4128, 1056),
    ((T128x256, 0, 0, 0), None, [2300], 2064, 2080),
]
PROGRAMS = {(0, 4, 4, 32), (0, 4, 8, 64), (0, 2, 8, 64), (0, 1, 8, 64), (0, 4, 4, 64), (T128, 0, 0, 0), (T256, 0, 0, 0),
            (T128x256, 0, 0, 0)}


def listed(shape):
    program, gated, counts, N, K = shape
    for g in (False, True) if gated is None else (gated,):
        for bf16 in (False, True):
            if not (program[0] == T128 and g and bf16):   # the gated BF16 product has no 128x128 tile
                yield (len(counts), sum(counts), N, K, int(g), int(bf16), 0, 0), program


@pytest.fixture(scope="module")
def program_of(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("programs") / "mxfp4_programs")
    subprocess.run(["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "dense_ragged_grouped_amd", "csrc"),
                    os.path.join(HERE, "mxfp4_programs.cpp"), "-o", exe], check=True)

    def ask(cases):
        text = "".join(" ".join(map(str, c)) + "\n" for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def test_the_shapes_reach_every_program(program_of):
    cases = [c for s in SHAPES for c in listed(s)]
    got = program_of([c for c, _ in cases])
    for (case, want), p in zip(cases, got):
        assert p == want, case
    assert set(got) == PROGRAMS


def test_limits_of_the_programs(program_of):
    """Codes leave in whole blocks of 32 columns; 128x128 tiles have room for 992 groups; a few-row launch stays below
    2^32 threads; a forced tile is taken where the product has it."""
    rng = np.random.default_rng(0)
    cases = []
    for _ in range(3000):
        E, M = int(rng.integers(1, 1025)), int(2 ** rng.uniform(0, 31))
        N, K = 16 * int(2 ** rng.uniform(0, 18)), 32 * int(2 ** rng.uniform(0, 17))
        cases.append((E, M, N, K, int(rng.integers(0, 2)), 0, 0, int(rng.choice([0, 0, 1, 2, 4]))))
    cases += [(*c[:4], 1, 0, 1, c[7]) for c in cases]
    for (E, M, N, K, gated, bf16, codes, tile), (t, nb, waves, tok) in zip(cases, program_of(cases)):
        if t == 0:
            assert tile == 0 or tile == T128 and E > 992
            assert nb == 4 or not codes
            blocks = (M // tok + min(M, E)) * -(-(N // 2 if gated else N) // (16 * (nb // 2 if gated else nb)))
            assert blocks * 64 * waves < 2 ** 32
        else:
            assert t in (T256, T128, T128x256) and (t != T128 or E <= 992)
            assert tile in (0, t) or tile == T128 and E > 992


# ---- on the GPU ----------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0][0]}-{s[0][1]}-{s[0][2]}-{s[0][3]}-{len(s[2])}x{s[3]}x{s[4]}")
def test_products(shape, gathered):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as drgg
    from tests.test_gpu_mxfp4 import check, counts_to_offsets, dev, gate64, grouped64, operand
    _, gated, counts, N, K = shape
    rng = np.random.default_rng(N + K)
    E, M = len(counts), sum(counts)
    T = M // 2 + 3 if gathered else M
    x, xs, xv = operand(rng, T, K, fill=254)
    w, ws, wv = operand(rng, E, N, K, fill=254)
    offsets = counts_to_offsets(counts)
    rows = None
    if gathered:
        rows = rng.integers(0, T, M).astype(np.int32)
        rows[::13] = -1
        xv = np.where((rows >= 0)[:, None], xv[rows], 0)
        rows = dev(rows)
    y, mag = grouped64(xv, wv, offsets, N)
    assert mag.max() * 64 < 2 ** 24
    for g in (False, True) if gated is None else (gated,):
        for dtype in (torch.float32, torch.bfloat16):
            got = drgg.grouped_gemm_mxfp4(x, xs, w, ws, dev(offsets), gated=g, rows=rows, out_dtype=dtype)
            if g:
                check(got, *gate64(y))
            else:
                assert torch.equal(got, dev(y).to(torch.float32).to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,I", [(3, 64, 2, 224, 288), (200, 64, 3, 96, 544), (1, 1, 1, 2080, 1056), (60, 4, 1, 576, 544),
                                       (350, 1, 1, 4128, 544), (80, 20, 9, 256, 544), (2400, 40, 1, 352, 544),
                                       (2300, 1, 1, 2080, 1056)])
def test_block_codes_in_every_program(T, E, k, H, I):
    """The activation's codes made in the first product's epilogue, in the programs that the rule takes for it."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as drgg
    from tests.test_gpu_mxfp4 import ffn_is_its_parts
    ffn_is_its_parts(drgg, T, E, k, H, I, False)
