"""Sizes past the 32-bit fields of the entry points' structures: refused, not wrapped around."""
import pytest
import torch

import kda_recurrent_state_amd as kda

WRAP = 1 << 32


def m(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


def t(*shape):
    return torch.zeros(*shape)


CASES = [
    ("num_seqs", lambda: kda.scan_fwd(t(4, 3), t(4, 3), num_seqs=WRAP + 1, final_state=False)),
    ("num_seqs", lambda: kda.scan_bwd(t(4, 3), t(4, 3), t(4, 3), num_seqs=WRAP + 2, initial_state_grad=False)),
    ("num_seqs", lambda: kda.conv_fwd(t(4, 3), t(3, 4), num_seqs=WRAP + 1, final_state=False)),
    ("num_seqs", lambda: kda.conv_bwd(t(4, 3), t(3, 4), t(4, 3), num_seqs=WRAP + 4, initial_state_grad=False)),
    ("num_seqs", lambda: kda.scan_workspace_size(t(4, 3), num_seqs=WRAP + 1)),
    ("num_seqs", lambda: kda.conv_bwd_workspace_size(t(4, 3), 4, num_seqs=1 << 31)),
    ("width", lambda: kda.conv_bwd_workspace_size(t(4, 3), WRAP + 4)),
    ("channels", lambda: kda.scan_fwd(m(1, WRAP + 8), m(1, WRAP + 8))),
    ("channels", lambda: kda.scan_step(m(1, WRAP + 8), m(1, WRAP + 8), m(1, WRAP + 8))),
    ("channels", lambda: kda.conv_fwd(m(1, WRAP + 8), m(WRAP + 8, 4))),
    ("width", lambda: kda.norm_gate_fwd(m(1, 1, WRAP + 8))),
    ("heads", lambda: kda.norm_gate_fwd(m(1, WRAP + 2, 4))),
    ("width", lambda: kda.residual_norm_fwd(m(1, WRAP + 8), m(1, WRAP + 8), m(WRAP + 8))),
    ("width", lambda: kda.residual_norm_bwd_workspace_size(m(1, WRAP + 8))),
    ("heads", lambda: kda.norm_gate_bwd_workspace_size(m(1, WRAP + 2, 4))),
    ("channels", lambda: kda.scan_workspace_size(m(1, WRAP + 8))),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_refused(i):
    name, f = CASES[i]
    with pytest.raises(ValueError, match=name + ".*32 bits"):
        f()
