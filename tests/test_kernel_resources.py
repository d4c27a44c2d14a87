"""Registers and LDS of the built kernels, from the metadata that the compiler
writes into the library: what the launchers and the planner assume about how
many workgroups share a compute unit (CPU only)."""
import os
import re
import shutil
import subprocess

import pytest

from tests.test_host import LIB, drgg  # noqa: F401  (the fixture that builds the library if there is none)

READELF = shutil.which("llvm-readelf") or os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin",
                                                       "llvm-readelf")
LDS_PER_CU, REGISTERS_PER_LANE = 160 * 1024, 512


@pytest.fixture(scope="module")
def kernels(drgg, tmp_path_factory):  # noqa: F811
    """{mangled name: {field: value}} of every kernel in the library's code objects."""
    if not os.path.exists(READELF):
        pytest.skip("needs llvm-readelf")
    data = open(LIB, "rb").read()
    found = {}
    for at in (m.start() for m in re.finditer(b"\x7fELF\x02\x01", data)):
        if int.from_bytes(data[at + 18:at + 20], "little") != 224:   # EM_AMDGPU
            continue
        part = tmp_path_factory.mktemp("objects") / f"{at}.o"
        part.write_bytes(data[at:])
        text = subprocess.run([READELF, "--notes", str(part)], capture_output=True, text=True, check=True).stdout
        for block in re.split(r"\n  - (?=\.)", text)[1:]:
            fields = dict(re.findall(r"\.(\w+):\s*(\d+)\n", block))
            name = re.search(r"\.symbol:\s*'?(\S+?)\.kd", block)
            if name:
                found[name.group(1)] = {k: int(v) for k, v in fields.items()}
    assert found
    return found


def per_cu(fields):
    """Workgroups that share a compute unit, by registers and by LDS: four SIMDs, registers in granules of 8."""
    waves = fields["max_flat_workgroup_size"] // 64
    per_simd = REGISTERS_PER_LANE // ((fields["vgpr_count"] + 7) // 8 * 8)
    return min(4 * per_simd // waves, LDS_PER_CU // fields["group_segment_fixed_size"])


def test_two_small_int8_tiles_share_a_cu(kernels):
    """launch_int8 starts 128x128 tiles two per CU and int8_tile prices them so: every variant has to fit, without scratch."""
    small = {n: f for n, f in kernels.items() if "int8_tile_kernelILi128ELi128E" in n}
    assert len(small) == 6
    for name, f in small.items():
        assert per_cu(f) == 2, (name, f)
        assert f["private_segment_fixed_size"] == 0 and f["vgpr_spill_count"] == 0, (name, f)


def test_no_kernel_spills(kernels):
    for name, f in kernels.items():
        assert f["vgpr_spill_count"] == 0 and f["private_segment_fixed_size"] == 0, (name, f)
