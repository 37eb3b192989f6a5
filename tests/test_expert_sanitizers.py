"""Host side of the expert feed-forward block (csrc/expert_api.cpp) under
AddressSanitizer and UndefinedBehaviorSanitizer on the CPU: built as plain C++
with the kernel launchers replaced by stubs that check their arguments
(tests/sanitize/expert_stubs.cpp) and driven through every entry point
(tests/sanitize/expert_driver.cpp)."""
import os

import pytest

from test_sanitizers import CLANG, ENV, ROOT, SAN, _check, _run


@pytest.mark.skipif(not os.path.exists(CLANG), reason="clang++ not available")
def test_expert_host_side_under_sanitizers(tmp_path):
    flags = ["-x", "c++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__",
             "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
             "-I" + os.path.join(ROOT, "combine_moe_layout_05_amd", "csrc"), *SAN]
    objs = []
    for src in (os.path.join(ROOT, "combine_moe_layout_05_amd", "csrc", "expert_api.cpp"),
                os.path.join(ROOT, "tests", "sanitize", "expert_stubs.cpp"),
                os.path.join(ROOT, "tests", "sanitize", "expert_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _check(_run([CLANG, *flags, "-c", src, "-o", obj]), f"compile {os.path.basename(src)}")
        objs.append(obj)
    exe = str(tmp_path / "expert_san")
    _check(_run([CLANG, *SAN[:1], *objs, "-o", exe]), "link")
    assert "0 failures" in _check(_run([exe], env=ENV), "run")
