"""Every program of the 8-bit product against exact integer products in 64
bits: the few-row programs' blocks of 16, 32 and 64 tokens and their K split,
and the tiles; with and without gathered rows and the gate, BF16 and FP32.

On the CPU: the shapes below run in the programs they are listed for, by the
launcher's own rule, and together reach every one.

Tolerances.  u = 2^-24: the sum is exact; its FP32 value and the two scales are
three roundings (4 u with second-order terms).  The gate's argument carries
those 4 u into exp, 4 |g| u, and exp, sum, reciprocal and products are within
16 u.  The output's rounding adds half the spacing of its type.
"""
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests.test_sanitize import HERE, ROOT, SAN

U = 2.0 ** -24
T256, T128, T128x256 = 1, 2, 4
MIXED = [0, 1, 16, 17, 32, 33, 15, 2, 31, 48]

# (program, gated or None for both, counts, N, K); program: (tile, nb, waves, tok)
SHAPES = [
    ((0, 4, 4, 32), None, (MIXED * 7)[:64], 528, 208),
    ((0, 4, 4, 32), None, (MIXED * 7)[:64], 528, 1040),
    ((0, 4, 4, 32), None, [0, 0, 70, 1] * 16, 560, 16),
    ((0, 4, 8, 64), None, [64, 33, 17, 16, 1, 0, 130, 48, 63, 20], 1040, 336),
    ((0, 4, 8, 64), None, [700], 1040, 4112),
    ((0, 2, 8, 64), None, [64, 33, 17, 16, 1, 0, 130], 1040, 560),
    ((0, 2, 8, 64), True, [65, 33, 16], 1040, 3088),
    ((0, 1, 8, 64), False, [65, 33, 16], 1040, 3088),
    ((0, 1, 8, 64), False, [1], 4096, 2064),
    ((0, 4, 4, 64), None, [64, 33, 17, 16, 1, 0, 62, 48, 63, 20, 130, 5, 31, 32, 49, 18, 40, 7, 65, 44], 1040, 256),
    ((0, 4, 4, 64), None, [400, 1, 300, 64, 190], 1472, 208),
    ((T128, 0, 0, 0), None, [60] * 40, 1040, 336),
    ((T256, 0, 0, 0), None, [300, 1, 4000, 257, 0, 6000], 2064, 144),
    ((T128x256, 0, 0, 0), None, [260] * 16, 1536, 2048),
]


def listed(shape):
    program, gated, counts, N, K = shape
    for g in (False, True) if gated is None else (gated,):
        for bf16 in (False, True):
            if not (program[0] == T128 and g and bf16):   # the gated BF16 product has no 128x128 tile
                yield (len(counts), sum(counts), N, K, int(g), int(bf16)), program


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_the_shapes_reach_every_program(tmp_path):
    exe = str(tmp_path / "int8_programs")
    subprocess.run(["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "dense_ragged_grouped_amd", "csrc"),
                    os.path.join(HERE, "int8_programs.cpp"), "-o", exe], check=True)
    cases = [c for s in SHAPES for c in listed(s)]
    text = "".join(" ".join(map(str, c)) + "\n" for c, _ in cases)
    got = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    for line, (case, want) in zip(got, cases):
        assert tuple(map(int, line.split())) == want, (case, line)
    for gated in (0, 1):
        reached = {p for c, p in cases if c[4] == gated}
        rows = {(0, 4, 4, 32), (0, 4, 8, 64), (0, 2, 8, 64), (0, 4, 4, 64)} | (set() if gated else {(0, 1, 8, 64)})
        assert reached == rows | {(t, 0, 0, 0) for t in (T256, T128, T128x256)}


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_long_groups_run_in_tiles(tmp_path):
    """Two blocks of 64 tokens per CU without more than 2048 rows a group: beyond, whatever K is, in tiles."""
    exe = str(tmp_path / "int8_programs")
    subprocess.run(["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "dense_ragged_grouped_amd", "csrc"),
                    os.path.join(HERE, "int8_programs.cpp"), "-o", exe], check=True)
    cases = [(1, 4793, 256, 4112), (1, 7673, 256, 2000), (1, 30713, 64, 144), (1, 1785, 1040, 400), (5, 1145, 1472, 2368),
             (16, 3321, 512, 784)]
    text = "".join(f"{E} {M} {N} {K} 0 1\n" for E, M, N, K in cases)
    got = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
    assert [int(t) != 0 for t in got[::4]] == [M > 2048 * E for E, M, _, _ in cases]


def product64(X, xs, W, ws, counts, gated):
    out, at = [], 0
    for e, n in enumerate(counts):
        y = X[at:at + n].astype(np.float64) @ W[e].astype(np.float64).T
        out.append(y * xs[at:at + n, None].astype(np.float64) * ws[e].astype(np.float64))
        at += n
    y = np.concatenate(out)
    if not gated:
        return y, 4 * U * np.abs(y)
    g, u = np.split(y, 2, axis=1)
    y = g / (1 + np.exp(-g)) * u
    return y, (4 * np.abs(g) + 16) * U * np.abs(y) + np.where(g < -80, np.abs(g * u) * 2.0 ** -100, 0) + 2.0 ** -126


@pytest.mark.gpu
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shape,gated", [(i, g) for i, s in enumerate(SHAPES)
                                         for g in ((False, True) if s[1] is None else (s[1],))])
def test_programs(shape, gated, bf16, gathered):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_ragged_grouped_amd as drgg
    _, _, counts, N, K = SHAPES[shape]
    E, M = len(counts), sum(counts)
    rng = np.random.default_rng(shape)
    T = M // 3 + 1 if gathered else M
    X, W = (rng.integers(-128, 128, s).astype(np.int8) for s in ((T, K), (E, N, K)))
    xs, ws = (rng.uniform(0.5, 2, s).astype(np.float32) / 64 for s in ((T,), (E, N)))
    if gated:   # gates of a few units
        xs = xs / np.float32(16 * np.sqrt(K))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = rng.integers(0, T, M).astype(np.int32) if gathered else np.arange(M)
    dtype = torch.bfloat16 if bf16 else torch.float32
    d = [torch.from_numpy(a).cuda() for a in (X, xs, W, ws, offsets)]
    out = torch.full((M + 2, N // 2 if gated else N), 7.0, dtype=dtype, device="cuda")
    drgg.grouped_gemm_int8(*d, gated=gated, rows=torch.from_numpy(rows).cuda() if gathered else None, out_dtype=dtype,
                           out=out[:M])
    want, before = product64(X[rows], xs[rows], W, ws, counts, gated)
    half = (2.0 ** -8 if bf16 else U) * np.exp2(np.floor(np.log2(np.maximum(np.abs(want) + before, 2.0 ** -126))))
    got = out[:M].float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= before + half)
    assert bool((out[M:] == 7.0).all())
