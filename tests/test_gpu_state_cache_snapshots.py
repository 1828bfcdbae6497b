"""The state layer's prefix states through the 8-bit cache: snapshots of a prefill into slots, read back as the states that
later prefills and decode steps start from, on one stream and in a captured graph."""
import numpy as np
import pytest
import torch

import kda_recurrent_state_amd as kda
from kda_recurrent_state_amd.workloads import WORKLOADS, generate, scaled
from oracle import kda_oracle
from tests import mixer_ref as M
from tests.parity import TOL, log, max_rel_err

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EVERY, LENGTHS = 64, [200, 64, 31, 0, 130]  # 3 + 1 + 0 + 0 + 2 snapshots
# the prefixes that the later requests go on from: row of the snapshots, tokens of their own
RESUMED = [(2, 50), (4, 1), (0, 64), (2, 7)]


def prefix_states(fmt, dtype, dv, seed):
    w = scaled(WORKLOADS["kda_varlen_64seq_h32_d128"], n_seqs=len(LENGTHS), heads=2, dk=64, dv=dv, dtype=dtype)
    inp = generate(w, seed=seed, device=DEV, lengths=LENGTHS)
    _, ST, snaps = kda.chunk_fwd_snapshots(inp["q"], inp["k"], inp["v"], inp["log_a"], inp["beta"], S0=inp["S0"],
                                           cu_seqlens=inp["cu_seqlens"], snapshot_every=EVERY)
    codes, scales = kda.state_cache_empty(9, snaps.shape[1:], fmt, DEV)
    slots = torch.tensor([7, 0, 3, 8, 1, 5], dtype=torch.int32, device=DEV)
    return snaps, ST, codes, scales, slots


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("dtype,dv", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 32)])
def test_resumed_from_the_cache(dtype, dv, fmt):
    log(f"snapshots through the cache {dtype} {dv} {fmt}")
    snaps, ST, codes, scales, slots = prefix_states(fmt, dtype, dv, 61)
    kda.state_cache_write(snaps, codes, scales, slots)
    want, ws = M.quantise(snaps.cpu(), fmt)
    at = slots.long()
    assert torch.equal(codes[at].float().cpu().double(), want) and torch.equal(scales[at].cpu(), ws)
    # a row is within half a step of its largest value: 1 / 254, and for e4m3 2^-4 of the value itself or 2^-10 of the scale
    held = want * ws.double()[..., None]
    near = snaps.cpu().double()
    step = near.abs().amax(-1, keepdim=True) / 254 if fmt == torch.int8 else \
        torch.maximum(near.abs() * 2.0 ** -4, ws.double()[..., None] * 2.0 ** -10)
    assert ((held - near).abs() <= step * (1 + 2.0 ** -20) + 2.0 ** -149).all()

    rows, lens = [r for r, _ in RESUMED], [n for _, n in RESUMED]
    pick = slots[torch.tensor(rows, device=DEV)].contiguous()
    S0 = kda.state_cache_read(codes, scales, pick)
    assert torch.equal(S0.cpu(), held.float()[rows])
    w = scaled(WORKLOADS["kda_varlen_64seq_h32_d128"], n_seqs=len(lens), heads=2, dk=64, dv=dv, dtype=dtype)
    inp = generate(w, seed=62, device=DEV, lengths=lens)
    o, S = kda.chunk_fwd(inp["q"], inp["k"], inp["v"], inp["log_a"], inp["beta"], S0=S0, cu_seqlens=inp["cu_seqlens"])
    ro, rS = kda_oracle(inp["q"], inp["k"], inp["v"], inp["log_a"], inp["beta"], S0=held[rows].numpy(),
                        cu_seqlens=inp["cu_seqlens"].cpu().numpy())
    e = max_rel_err(o, ro), max_rel_err(S, rS)
    # and one token more, from the states as they are kept
    last = torch.cumsum(torch.tensor(lens), 0) - 1
    one = {k: inp[k][last].contiguous() for k in ("q", "k", "v", "log_a", "beta")}
    kda.state_cache_write(S, codes, scales, pick.new_tensor([2, 4, 6, 2]))
    kept = kda.state_cache_read(codes, scales, pick.new_tensor([2, 4, 6, 2]))
    assert torch.equal(kept[0], kept[3])
    want, ws = M.quantise(S.cpu()[[3, 1, 2, 3]], fmt)
    assert torch.equal(kept.cpu(), want.float() * ws[..., None])
    ot, _ = kda.decode_step(one["q"], one["k"], one["v"], one["log_a"], one["beta"], kept.clone())
    ro, _ = kda_oracle(one["q"], one["k"], one["v"], one["log_a"], one["beta"], S0=kept.cpu().double().numpy(),
                       cu_seqlens=np.arange(len(lens) + 1))
    e += (max_rel_err(ot, ro),)
    log("  err " + " ".join(f"{x:.2e}" for x in e))
    assert max(e) <= TOL[dtype]


def test_in_a_graph():
    """Snapshots written, read and resumed from in one captured graph, replayed with eager work between."""
    log("snapshots through the cache in a graph")
    snaps, ST, codes, scales, slots = prefix_states(torch.int8, torch.bfloat16, 128, 63)
    rows, lens = [r for r, _ in RESUMED], [n for _, n in RESUMED]
    pick = slots[torch.tensor(rows, device=DEV)].contiguous()
    w = scaled(WORKLOADS["kda_varlen_64seq_h32_d128"], n_seqs=len(lens), heads=2, dk=64, dv=128)
    inp = generate(w, seed=64, device=DEV, lengths=lens)
    S0 = torch.empty((len(rows),) + tuple(snaps.shape[1:]), device=DEV)

    def work():
        kda.state_cache_write(snaps, codes, scales, slots)
        kda.state_cache_read(codes, scales, pick, out=S0)
        return kda.chunk_fwd(inp["q"], inp["k"], inp["v"], inp["log_a"], inp["beta"], S0=S0, cu_seqlens=inp["cu_seqlens"],
                             max_seqlen=max(lens))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = work()
    for i in range(3):
        snaps.mul_(1.5 if i else 1.0)
        codes.zero_(), scales.zero_(), S0.zero_(), o.zero_(), S.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), S.clone(), codes.clone(), scales.clone()
        want = work()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got[2], codes) and torch.equal(got[3], scales)
