"""The largest accepted sizes fit one launch (CPU only): tests/sanitize/launch_limits.cpp,
and the refusal through the library."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_launch_limits(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not installed")
    exe = str(tmp_path / "launch_limits")
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-Wall", "-o", exe,
                           os.path.join(ROOT, "tests", "sanitize", "launch_limits.cpp")])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "launch limits ok" in r.stdout, r.stderr


@pytest.mark.parametrize("R", [(1 << 30) - 63, (1 << 30) - 1, 1 << 30])
def test_rows_past_one_launch_are_refused(R):
    from speculative_sampling_verification_vocab_amd import _native
    p = ctypes.c_void_p
    st = _native.load().spec_quantize_rows(p(0x1000), R, 1, _native.SPEC_BF16, p(0x2000), p(0x3000), None)
    assert st == 2   # unsupported, before anything is launched
