"""Sizes of zero in the state space scan's, the gated products' and the state cache's calls: an error of the binding's or of
the library's, nothing else, and nothing launched (CPU)."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests.test_mixer_boundary_cpu import f, launched  # noqa: F401

ZERO = [("heads", 0), ("groups", 1), ("state", 2), ("width", 3)]


def sizes(i):
    s = [4, 2, 8, 6]
    s[i] = 0
    return s


@pytest.mark.parametrize("name,i", ZERO)
@pytest.mark.parametrize("fn", ["ssm_fwd", "ssm_bwd", "ssm_conv_step", "ssm_workspace_size",
                                "ssm_conv_step_workspace_size"])
def test_scan(launched, fn, name, i):  # noqa: F811
    H, G, K, P = sizes(i)
    N, T = 2, 2
    ch = H * P + 2 * G * K
    base = dict(x=f(T, H, P), dt=f(T, H), A=f(H), B=f(T, G, K), C=f(T, G, K))
    calls = {"ssm_fwd": lambda: kda.ssm_fwd(**base), "ssm_bwd": lambda: kda.ssm_bwd(**base, dy=f(T, H, P)),
             "ssm_conv_step": lambda: kda.ssm_conv_step(f(N, ch), f(ch, 4), f(N, 3, ch), f(N, H), f(H), f(N, H, K, P)),
             "ssm_workspace_size": lambda: kda.ssm_workspace_size(f(T, H, P), f(T, G, K)),
             "ssm_conv_step_workspace_size": lambda: kda.ssm_conv_step_workspace_size(f(N, ch), f(N, H, K, P))}
    with pytest.raises((ValueError, kda.KdaError), match="channels" if name == "groups" and "conv" in fn else None):
        calls[fn]()
    assert not launched


@pytest.mark.parametrize("shape,w", [((4, 0), (3, 0)), ((4, 8), (0, 8))], ids=["width", "hidden"])
def test_products(launched, shape, w):  # noqa: F811
    for call in (lambda: kda.glu_fwd(f(*shape), f(*w), f(*w)), lambda: kda.glu_bwd(f(*shape), f(*w), f(*w), f(4, w[0])),
                 lambda: kda.glu_workspace_size(f(*shape), f(*w), f(*w))):
        with pytest.raises((ValueError, kda.KdaError)):
            call()
    assert not launched


def test_a_conv_step_of_no_state_rows_says_so():
    with pytest.raises(ValueError, match="state rows"):
        kda.ssm_conv_step_workspace_size(f(2, 24), torch.zeros(2, 4, 0, 6))
