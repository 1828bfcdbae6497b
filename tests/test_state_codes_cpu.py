"""The quotient behind the state cache's codes, on the host (CPU)."""
from tests.test_scan_launch_cpu import host_check


def test_quotients_lie_on_their_side_of_every_border(tmp_path):
    assert "state codes check ok" in host_check("state_codes_check", tmp_path)
