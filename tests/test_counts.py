"""The numbers of tiles and chunks of a group of up to 2^31 - 1 rows, as the
kernels compute them, under the host's sanitizers; and on the GPU the products
at that length."""
import os
import shutil
import subprocess

import pytest

from tests.test_sanitize import HERE, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_counts_of_the_longest_groups(tmp_path):
    exe = str(tmp_path / "counts_driver")
    subprocess.run(["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "dense_ragged_grouped_amd", "csrc"),
                    os.path.join(HERE, "counts_driver.cpp"), "-o", exe], check=True)
    _run(exe, tmp_path)


MOST = 2 ** 31 - 1


@pytest.fixture
def memory():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free memory")
    yield torch
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_int8_product_of_the_most_rows(memory):
    """One group of 2^31 - 1 rows: the first and the last rows as in small calls, all rows written."""
    import dense_ragged_grouped_amd as drgg
    torch, (N, K) = memory, (8, 16)
    q = torch.empty((MOST, K), dtype=torch.int8, device="cuda").random_(-127, 128)
    s = torch.ones(MOST, device="cuda")
    w = torch.randint(-127, 128, (N, K), device="cuda", dtype=torch.int32).to(torch.int8)
    ws = torch.ones(N, device="cuda")
    out = torch.full((MOST, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    drgg.gemm_int8(q, s, w, ws, out=out)
    for part in (slice(0, 700), slice(MOST // 2, MOST // 2 + 700), slice(MOST - 700, MOST)):
        assert torch.equal(out[part], drgg.gemm_int8(q[part], s[part].clone(), w, ws))
    for lo in range(0, MOST, 1 << 28):
        assert not bool(out[lo:lo + (1 << 28), 0].isnan().any())


@pytest.mark.gpu
def test_bf16_product_of_the_most_rows(memory):
    import dense_ragged_grouped_amd as drgg
    torch, (N, K) = memory, (8, 8)
    x = torch.empty((MOST, K), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.randn((1, N, K), device="cuda").to(torch.bfloat16)
    out = torch.full((MOST, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    drgg.grouped_gemm_fwd(x, w, torch.tensor([0, MOST], dtype=torch.int32, device="cuda"), out=out)
    few = torch.tensor([0, 700], dtype=torch.int32, device="cuda")
    for part in (slice(0, 700), slice(MOST // 2, MOST // 2 + 700), slice(MOST - 700, MOST)):
        assert torch.equal(out[part], drgg.grouped_gemm_fwd(x[part], w, few))
    for lo in range(0, MOST, 1 << 28):
        assert not bool(out[lo:lo + (1 << 28), 0].isnan().any())
