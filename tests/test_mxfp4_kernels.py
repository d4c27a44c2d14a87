"""The 4-bit products' kernels in the built library (CPU only): none that no call
reaches.  Codes and scales leave only the serving block's first product, which gathers
its rows by token."""
import re

from tests.test_host import drgg  # noqa: F401  (the fixture that builds the library if there is none)
from tests.test_kernel_resources import kernels  # noqa: F401

CODES = 2   # MxOut: FP32 and BF16 values, codes


def test_codes_leave_gathered_products_alone(kernels):  # noqa: F811
    """Template arguments in the names: result (an enumerator), gated, gathered, behind the tile's two sizes."""
    found = [(n, re.search(r"mx_(rows|tile)_kernelI(?:Li\d+ELi\d+E)?L\w+?E(\d)ELb(\d)ELb(\d)E", n)) for n in kernels
             if re.search(r"mx_(rows|tile)_kernel", n)]
    assert found and all(m for _, m in found)
    codes = [m.groups() for _, m in found if int(m.group(2)) == CODES]
    assert {kind for kind, *_ in codes} == {"rows", "tile"}
    assert all((gated, gathered) == ("1", "1") for _, _, gated, gathered in codes), codes
