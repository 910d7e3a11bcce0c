"""Rules that the CUDA sources keep and no run can show: what breaks them gives
right results nearly always."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemv_zero_point_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_inputs_of_early_kernels_are_not_read_as_constants():
    """A kernel that is resident while the work before it writes its inputs
    reads them by ordinary loads: loads of constants (__ldg, or a const
    __restrict__ parameter, which lets the compiler choose them) are defined
    for data that nobody writes during the kernel's life."""
    rows = _code("expert_rows.cu")
    assert "griddepcontrol.wait" in rows
    assert "__ldg" not in rows and ".nc" not in rows
    assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", rows)
    gather = _code("a16w4_tc.cu")
    gather = gather[gather.index("a16w4_gather_kernel(const"):gather.index("g_tc_encode = nullptr")]
    assert "griddepcontrol.wait" in gather and "__ldg" not in gather
    assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", gather)
