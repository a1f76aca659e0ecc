"""The packed sequences' search under UndefinedBehaviorSanitizer (host build, CPU only)."""
import os
import shutil

import pytest

from tests.test_sanitize import HERE, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_search_over_up_to_the_most_sequences(tmp_path):
    rocm, exe = os.environ.get("ROCM_PATH", "/opt/rocm"), str(tmp_path / "sequence_check")
    rc, out = _run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-g", "-O1",
                    "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"), os.path.join(HERE, "sequence_check.cpp"), "-o", exe])
    assert rc == 0, out
    rc, out = _run([exe])
    print(out)
    assert rc == 0 and (out.startswith("ok") or out.startswith("skipped")), out
