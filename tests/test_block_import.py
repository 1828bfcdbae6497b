"""The package on a torch without the quick way to the current stream's handle."""
import os
import subprocess
import sys

import pytest
import torch

import kda_recurrent_state_amd as kda
from kda_recurrent_state_amd import block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_the_quick_stream_handle():
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import kda_recurrent_state_amd as kda\n"
            "t = torch.zeros(4, 3)\n"
            "try: kda.scan_fwd(t, t)\n"
            "except RuntimeError as e: print('refused:', e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "refused:" in r.stdout


@pytest.mark.gpu
def test_stream_handles_agree():
    """Both ways name the current stream, and a call made the other way runs on it."""
    x, la = torch.randn(300, 6, device="cuda:0"), -torch.rand(300, 6, device="cuda:0")
    want = kda.scan_fwd(x, la)[0]
    quick = block._raw_stream
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert block._stream_of(0) == quick(0) == s.cuda_stream
        block._raw_stream = block._stream_of
        try:
            got = kda.scan_fwd(x, la)[0]
        finally:
            block._raw_stream = quick
    torch.cuda.synchronize()
    assert torch.equal(got, want)
