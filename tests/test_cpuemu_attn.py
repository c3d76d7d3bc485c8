"""The attention and cache kernels on the CPU, before any GPU run: the same
emulation and guard pages as test_cpuemu.py (matrix instructions and the
transposing LDS read included), compared with 64-bit references within
tolerances counted in roundings (tests/attn_ref.py)."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CASES = os.path.join(HERE, "cpuemu", "attn_cases.py")


@pytest.fixture(scope="module")
def emu_lib():
    sys.path.insert(0, os.path.join(HERE, "cpuemu"))
    try:
        import build as emu_build
        return emu_build.build()
    finally:
        sys.path.pop(0)


@pytest.mark.parametrize("place", ["end", "start"])
@pytest.mark.parametrize("family", ["prompt", "decode", "pages"])
def test_kernels_on_guarded_buffers(emu_lib, family, place):
    env = dict(os.environ, EMU_CUS="4")
    r = subprocess.run([sys.executable, CASES, family, place], capture_output=True, text=True, env=env,
                       timeout=900)
    tail = "\n".join((r.stdout + r.stderr).strip().splitlines()[-8:])
    assert r.returncode == 0, f"{family}/{place} exited with {r.returncode}:\n{tail}"
    assert "all cases passed" in r.stdout, tail
