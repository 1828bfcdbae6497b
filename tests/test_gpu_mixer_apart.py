"""States updated in place on the GPU: refused on another tensor of the call, with nothing changed, and accepted between the
tokens of a tensor whose tokens lie apart."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests.parity import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
N, H, G, K, P, W = 3, 4, 2, 16, 8, 4
CH = H * P + 2 * G * K


def rand(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(DEV)


def step_args():
    return dict(x=rand(N, H, P, seed=1), dt=rand(N, H, seed=2), A=-rand(H, seed=3).abs(), B=rand(N, G, K, seed=4),
                C=rand(N, G, K, seed=5), h=rand(N, H, K, P, seed=6), D=rand(H, seed=7), dt_bias=rand(H, seed=8))


def conv_args():
    a = step_args()
    return dict(xbc=rand(N, CH, seed=9), conv_weight=rand(CH, W, seed=10), conv_state=rand(N, W - 1, CH, seed=11), dt=a["dt"],
                A=a["A"], h=a["h"], D=a["D"], dt_bias=a["dt_bias"], conv_bias=rand(CH, seed=12))


CASES = [(kda.ssm_step, step_args, "h", n) for n in ("x", "dt", "A", "B", "C", "D", "dt_bias")] + \
    [(kda.ssm_conv_step, conv_args, s, n) for s in ("h", "conv_state")
     for n in ("xbc", "conv_weight", "dt", "A", "D", "dt_bias", "conv_bias", "conv_state") if n != s]


@pytest.mark.parametrize("fn,make,state,name", CASES, ids=lambda v: getattr(v, "__name__", str(v)))
def test_refused(fn, make, state, name):
    log(f"{fn.__name__}: {state} updated in place on {name}")
    a = make()
    fn(**a)
    a = make()
    big = torch.zeros(a[state].numel() + a[name].numel(), device=DEV)
    at = a[state].numel() - 1  # one value is both's
    big[at:at + a[name].numel()] = a[name].flatten()
    a[state], a[name] = big[:a[state].numel()].view(a[state].shape), big[at:at + a[name].numel()].view(a[name].shape)
    before = big.clone()
    with pytest.raises(kda.KdaError, match="overlaps"):
        fn(**a)
    assert torch.equal(big, before)


def test_between_tokens():
    """x's tokens far apart, and the state between the first two of them."""
    log("ssm_step: h between the tokens of x")
    a = step_args()
    want = kda.ssm_step(**step_args())
    wide = H * P + a["h"].numel()
    store = torch.zeros(N, wide, device=DEV)
    store[:, :H * P] = a["x"].flatten(1)
    h = store.view(-1)[H * P:wide].view(a["h"].shape)
    h.copy_(a["h"])
    y, ho = kda.ssm_step(**{**a, "x": store[:, :H * P].view(N, H, P), "h": h})
    assert ho is h and torch.equal(y, want[0]) and torch.equal(ho, want[1])
    assert torch.equal(store[:, :H * P].reshape(N, H, P), a["x"])
