"""The scan's launch, on the host: the sizes at which it would be too large, and which of its
threads publish a channel's state."""
import os

import pytest

import kda_recurrent_state_amd as kda
from tests.test_block_boundary_cpu import INVALID, call, scan_dims
from tests.test_sanitizers_cpu import HIPCC, ROOT, SAN, _run

LAST = 1073725184  # the last T of up to 64 channels: its 4194239 tiles and 64 more workgroups of 1024 threads are 2^32 - 1024


@pytest.mark.parametrize("fn", ["kda_scan_fwd", "kda_scan_bwd"])
@pytest.mark.parametrize("T", [LAST + 1, LAST + 2000, 1073733504])
@pytest.mark.parametrize("C", [1, 2, 64])
def test_room_for_the_empty_sequences(fn, T, C):
    """Tiles of 256 tokens take 1024 threads, and up to 64 workgroups more hand empty
    sequences their states: a call whose launch would pass 2^32 threads is refused."""
    lib = kda.load_library()
    assert (-(-T // 256) + 64) * 1024 >= 1 << 32
    assert call(lib, fn, scan_dims(num_seqs=64, total_tokens=T, channels=C)) == INVALID
    assert "too large" in lib.kda_last_error().decode()


def host_check(name, tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / name)
    _run([HIPCC, "-x", "hip", "-O1", "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
          "-packed-fp32-ops", "-I" + os.path.join(ROOT, "kda_recurrent_state_amd", "csrc"),
          os.path.join(SAN, name + ".cpp"), "-o", exe])
    return _run([exe]).stdout


def test_accepted_sizes_fit_a_launch(tmp_path):
    assert "scan launch check ok" in host_check("scan_launch_check", tmp_path)


def test_one_publisher_for_each_channel(tmp_path):
    """In rows of odd length a block's end lane moves back by a column, which its neighbour
    (of the next workgroup's wavefront, or of another) owns: only that one publishes it."""
    assert "scan owner check ok" in host_check("scan_owner_check", tmp_path)
