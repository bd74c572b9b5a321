"""AddressSanitizer / UndefinedBehaviorSanitizer run of the host half of the
8-bit operators and the token log-probabilities (CPU only):
tests/sanitize/host_checks_quant.cpp, built with gcc and with ROCm's clang."""
import os
import subprocess

import pytest

from tests.test_sanitizers import COMPILERS, ROOT, SAN, _available, _run


@pytest.mark.parametrize("compiler", sorted(COMPILERS))
def test_host_checks_under_sanitizers(compiler, tmp_path):
    cxx = COMPILERS[compiler][1]
    if not _available(cxx):
        pytest.skip(f"{cxx} not installed")
    exe = str(tmp_path / "host_checks_quant")
    subprocess.check_call([cxx, "-std=c++17", *SAN, "-Wall", "-o", exe,
                           os.path.join(ROOT, "tests", "sanitize", "host_checks_quant.cpp")])
    rc, out, err = _run(exe)
    assert rc == 0 and "host checks ok" in out, err[-4000:]
    assert "runtime error" not in err and "ERROR: AddressSanitizer" not in err, err[-4000:]
