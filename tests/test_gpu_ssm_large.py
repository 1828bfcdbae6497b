"""The state space scan's gradient over more than 2^32 bytes of inputs and of states kept by chunk, one workgroup to all of a
group's units: every gradient against the calls of its sequences alone."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests.parity import log
from tests.test_gpu_mixer_large import ssm_inputs

pytestmark = pytest.mark.gpu


def test_every_gradient_of_more_than_32_bits():
    log("ssm gradient 2^32 bytes")
    N, L, H, P, K = 70, 512, 64, 1024, 16
    v = ssm_inputs(N * L, N, H, 1, K, P, torch.bfloat16)
    dy = v["x"].flip(0)
    got = kda.ssm_bwd(**v, dy=dy, num_seqs=N)
    assert v["x"].nbytes > 1 << 32 and N * L // 64 * H * 32 * P * 4 > 1 << 32  # states are kept in blocks of 32 rows
    total, mag = {}, {}
    for n in range(N):
        t = slice(n * L, (n + 1) * L)
        one = dict(v, **{k: v[k][t].clone() for k in ("x", "dt", "B", "C")}, h0=v["h0"][n:n + 1].clone())
        g = kda.ssm_bwd(**one, dy=dy[t].clone())
        for k in ("dx", "dB", "dC"):
            # both within a half step of their type; sums in another order: up to 4096 additions of partial sums of up
            # to 4 times the largest, 2^-10 of it
            a, b = got[k][t].float(), g[k].float()
            assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -10 * b.abs().max()).all(), (n, k)
        for k, a in (("ddt", got["ddt"][t]), ("dh0", got["dh0"][n:n + 1])):
            assert ((a - g[k]).abs() <= 2.0 ** -10 * g[k].abs().max()).all(), (n, k)
        for k in ("dA", "dD", "ddt_bias"):
            total[k] = total.get(k, 0) + g[k].double()
            mag[k] = mag.get(k, 0) + g[k].double().abs()
    for k in total:  # a sequence lost or taken twice would be a seventieth
        assert ((got[k].double() - total[k]).abs() <= 2.0 ** -14 * (mag[k] + mag[k].max())).all(), k
