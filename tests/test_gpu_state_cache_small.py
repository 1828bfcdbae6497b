"""The 8-bit state cache where quotients are far below the scale, on the GPU against exact arithmetic
(tests/mixer_ref.py): codes and scales have to be equal."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_ref as M
from tests.parity import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMATS = [torch.int8, torch.float8_e4m3fn]


def same_codes(rows, fmt):
    """rows [R, W] float32, each a state of one row."""
    x = rows[:, None]
    codes, scales = kda.state_cache_empty(x.shape[0], x.shape[1:], fmt, DEV)
    kda.state_cache_write(x.to(DEV), codes, scales)
    want, ws = M.quantise(x, fmt)
    assert torch.equal(scales.cpu(), ws)
    assert torch.equal(codes.float().cpu().double(), want)
    back = kda.state_cache_read(codes, scales).cpu()
    assert torch.equal(back, want.float() * ws[..., None])


@pytest.mark.parametrize("fmt", FORMATS)
def test_quotients_that_underflow(fmt):
    """Values whose quotient is zero in float32, of both signs, beside one below every border (which has the lane's four
    divided), in each place of the four."""
    log(f"state cache, quotients that underflow {fmt}")
    rows = []
    for most in (1000.0, 1e10, 3e38, 1.0):
        for tiny in (2.0 ** -149, 1.2e-38, 2.0 ** -126, 2.0 ** -140):
            for small in (1e-5, 1e-7):
                quad = [most * small, tiny, -tiny, 0.0]
                for k in range(4):
                    rows.append([most, 0.0, 0.0, 0.0] + quad[k:] + quad[:k])
                rows.append([most, most * small, tiny, -tiny] + [0.0] * 4)
    same_codes(torch.tensor(rows, dtype=torch.float32), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_borders_of_small_scales(fmt):
    """Values on and beside the middles between neighbouring codes where the scale is the least number, subnormal or
    just above, so that the quotient's remainder is below what float32 holds."""
    log(f"state cache, borders of small scales {fmt}")
    values, _ = M.formats(fmt)
    mid = (values[1:] + values[:-1]) / 2
    rows = []
    for s in (2.0 ** -149, 2.0 ** -140 + 2.0 ** -149, 2.0 ** -126, 2.0 ** -126 + 2.0 ** -149, 1.7 * 2.0 ** -126, 1.1 * 2.0 ** -125,
              1.3 * 2.0 ** -120, 1.9 * 2.0 ** -61):
        most = (values[-1] * s).float()
        v = (mid * s).float()
        for step in range(-3, 4):
            w = v.clone()
            for _ in range(abs(step)):
                w = torch.nextafter(w, torch.full_like(w, 1.0 if step > 0 else -1.0))
            rows.append(torch.cat([w, most[None]]))
    same_codes(torch.stack(rows), fmt)
