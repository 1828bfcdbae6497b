"""CPU-only sanitizer build (AddressSanitizer and UndefinedBehaviorSanitizer) of the host side
of the state space scan, the gated feed-forward products and the state cache, driven by
tests/sanitize/mixer_check.cpp with calls that the host refuses or that have nothing to do.
No GPU is used."""
import os

import pytest

from tests.test_sanitizers_cpu import BUILD, ENV, HIPCC, ROOT, SAN, _check_clean, _run

APIS = ("kda_ssm_api.cpp", "kda_glu_api.cpp", "kda_state_cache_api.cpp")


def test_mixer_host_validation_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from kda_recurrent_state_amd import _build
    objs = [os.path.join(BUILD, os.path.splitext(f)[0] + ".o") for f in _build.SOURCES if f not in APIS]
    if not all(os.path.exists(o) for o in objs):
        _build.build()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all"]
    apis = [str(tmp_path / (a + ".o")) for a in APIS]
    chk_o, exe = str(tmp_path / "check.o"), str(tmp_path / "mixer_check")
    for src, obj in zip(APIS, apis):
        _run([HIPCC, "-x", "hip", "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *san, "-I" + os.path.join(ROOT, "include"),
              "-c", os.path.join(_build.CSRC, src), "-o", obj])
    _run([HIPCC, "-O1", "-g", "-std=c++17", *san, "-I" + os.path.join(ROOT, "include"),
          "-c", os.path.join(SAN, "mixer_check.cpp"), "-o", chk_o])
    _run([HIPCC, "--offload-arch=gfx950", *san, chk_o, *apis, *objs, "-o", exe])
    r = _run([exe], env=ENV)
    _check_clean(r)
    assert "mixer api sanitizer check ok" in r.stdout
