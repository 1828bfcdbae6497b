"""CPU-only sanitizer build (AddressSanitizer and UndefinedBehaviorSanitizer) of
the host side of the operators around the state layer (kda_block_api.cpp),
driven by tests/sanitize/block_check.cpp with calls that the host refuses or
that have nothing to do.  No GPU is used."""
import os

import pytest

from tests.test_sanitizers_cpu import BUILD, ENV, HIPCC, ROOT, SAN, _check_clean, _run


def test_block_host_validation_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from kda_recurrent_state_amd import _build
    objs = [os.path.join(BUILD, os.path.splitext(f)[0] + ".o") for f in _build.SOURCES if f != "kda_block_api.cpp"]
    if not all(os.path.exists(o) for o in objs):
        _build.build()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all"]
    api_o, chk_o, exe = (str(tmp_path / n) for n in ("api.o", "check.o", "block_check"))
    _run([HIPCC, "-x", "hip", "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *san, "-I" + os.path.join(ROOT, "include"),
          "-c", os.path.join(_build.CSRC, "kda_block_api.cpp"), "-o", api_o])
    _run([HIPCC, "-O1", "-g", "-std=c++17", *san, "-I" + os.path.join(ROOT, "include"),
          "-c", os.path.join(SAN, "block_check.cpp"), "-o", chk_o])
    _run([HIPCC, "--offload-arch=gfx950", *san, chk_o, api_o, *objs, "-o", exe])
    r = _run([exe], env=ENV)
    _check_clean(r)
    assert "block api sanitizer check ok" in r.stdout
