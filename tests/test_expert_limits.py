"""CPU tests of the expert block's largest sizes."""
import os

import pytest

from test_sanitizers import CLANG, ENV, ROOT, SAN, _check, _run


@pytest.mark.skipif(not os.path.exists(CLANG), reason="clang++ not available")
def test_row_counts_up_to_the_largest(tmp_path):
    """The division of a segment into tiles and steps stays within 32 bits
    (tests/sanitize/expert_limits.cpp, under UndefinedBehaviorSanitizer)."""
    exe = str(tmp_path / "limits")
    _check(_run([CLANG, "-x", "c++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__",
                 "-I/opt/rocm/include",
                 "-I" + os.path.join(ROOT, "combine_moe_layout_05_amd", "csrc"), *SAN,
                 os.path.join(ROOT, "tests", "sanitize", "expert_limits.cpp"), "-o", exe]),
           "compile")
    assert "0 failures" in _check(_run([exe], env=ENV), "run")
