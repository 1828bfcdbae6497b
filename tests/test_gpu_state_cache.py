"""The 8-bit state cache on the GPU against exact arithmetic (tests/mixer_ref.py): codes and scales have to be equal."""
import pytest
import torch

import kda_recurrent_state_amd as kda
from tests import mixer_ref as M

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMATS = [torch.int8, torch.float8_e4m3fn]
SHAPES = [(2, 16, 128), (3, 7, 83), (1, 5, 1), (1, 4, 3), (2, 3, 4), (1, 2, 257), (1, 3, 1500), (1, 2, 8192), (40,)]


def states_of(R, shape, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, *shape, generator=g) * torch.exp(2 * torch.randn(R, *shape[:-1], 1, generator=g))
    if shape[-1] > 2:
        x[0, ..., 1] = -x[0].abs().amax(-1)  # the largest magnitude twice, once negative
    return x


def raw(codes):
    return codes.view(torch.int8)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_round_trip(shape, fmt):
    x = states_of(4, shape, 1)
    x[2] = 0
    codes, scales = kda.state_cache_empty(6, shape, fmt, DEV)
    slots = torch.tensor([5, 0, 3, 2], dtype=torch.int32, device=DEV)
    kda.state_cache_write(x.to(DEV), codes, scales, slots)
    want, ws = M.quantise(x, fmt)
    at = slots.long().cpu()
    assert torch.equal(scales.cpu()[at], ws)
    assert torch.equal(codes.float().cpu()[at].double(), want)
    assert not raw(codes)[[1, 4]].any() and not scales[[1, 4]].any()
    back = kda.state_cache_read(codes, scales, slots)
    assert torch.equal(back.cpu(), want.float() * ws[..., None])
    assert torch.equal(kda.state_cache_read(codes, scales)[at.to(DEV)], back)
    assert torch.equal(kda.state_cache_read(codes, scales, slots, out=torch.full_like(back, 9.0)), back)


@pytest.mark.parametrize("fmt", FORMATS)
def test_borders(fmt):
    """Values on and beside the middles between neighbouring codes, for scales whose quotients are not exact."""
    values, _ = M.formats(fmt)
    mid = ((values[1:] + values[:-1]) / 2).float()
    most = values[-1].float()
    rows = []
    for s in (1.0, 1.1, 0.7, 3.3e-5, 777.7, 1.9e30, 2.3e-30):
        s = torch.tensor(s, dtype=torch.float32)
        m = mid * s
        for v in (m, torch.nextafter(m, m + s), torch.nextafter(m, m - s)):
            rows.append(torch.cat([v, (most * s)[None]]))
    x = torch.stack(rows)[:, None]
    codes, scales = kda.state_cache_empty(len(rows), x.shape[1:], fmt, DEV)
    kda.state_cache_write(x.to(DEV), codes, scales)
    want, ws = M.quantise(x, fmt)
    assert torch.equal(scales.cpu(), ws)
    assert torch.equal(codes.float().cpu().double(), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_special_rows(fmt):
    """Zeros, the smallest and largest numbers, an infinity, a NaN."""
    W = 8
    x = torch.zeros(7, W)
    x[1, 0] = 2.0 ** -149
    x[2, :3] = torch.tensor([2.0 ** -140, -2.0 ** -141, 2.0 ** -149])
    x[3, :2] = torch.tensor([3.4e38, -1.7e38])
    x[4, 0], x[4, 1] = float("inf"), 1.0
    x[5, 3] = float("nan")
    x[6] = -0.0
    codes, scales = kda.state_cache_empty(1, (7, W), fmt, DEV)
    kda.state_cache_write(x[None].to(DEV), codes, scales)
    back = kda.state_cache_read(codes, scales).cpu()[0]
    assert (back[0] == 0).all() and (back[6] == 0).all() and torch.isfinite(back[1:4]).all()
    assert torch.isnan(back[4]).all() and torch.isnan(back[5]).all()
    step = 1 / 254 if fmt == torch.int8 else 2.0 ** -4
    assert ((back[3] - x[3]).abs() <= 1.01 * step * 3.4e38).all()
    # a scale in the subnormal range is held to 2^-149, a code of 127 or 448 steps of it to so many
    assert ((back[1:3] - x[1:3]).abs() <= 448 * 2.0 ** -149).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_slots(fmt):
    """A slot named twice keeps the last state; slots outside the cache are skipped, and read as zeros."""
    shape = (3, 20)
    x = states_of(9, shape, 2)
    slots = [2, -1, 2, 5, 7, 2, 100, 0, 5]
    codes, scales = kda.state_cache_empty(7, shape, fmt, DEV)
    raw(codes).fill_(3)
    scales.fill_(2.0)
    sd = torch.tensor(slots, dtype=torch.int32, device=DEV)
    kda.state_cache_write(x.to(DEV), codes, scales, sd)
    want, ws = M.quantise(x, fmt)
    for slot, r in ((2, 5), (5, 8), (0, 7)):
        assert torch.equal(codes[slot].float().cpu().double(), want[r]) and torch.equal(scales[slot].cpu(), ws[r])
    for slot in (1, 3, 4, 6):
        assert (raw(codes)[slot] == 3).all() and (scales[slot] == 2).all()
    back = kda.state_cache_read(codes, scales, sd)
    for i, s in enumerate(slots):
        if 0 <= s < 7:
            assert torch.equal(back[i], codes[s].float() * scales[s][..., None])
        else:
            assert not back[i].any()


def test_many_states():
    """More states than a launch has workgroups for one block of rows each, with repeated slots."""
    R, shape = 9000, (2, 8)
    x = torch.randn(R, *shape, generator=torch.Generator().manual_seed(3))
    slots = torch.randint(0, 5000, (R,), generator=torch.Generator().manual_seed(4)).to(torch.int32)
    codes, scales = kda.state_cache_empty(5000, shape, torch.int8, DEV)
    kda.state_cache_write(x.to(DEV), codes, scales, slots.to(DEV))
    want, ws = M.quantise(x, torch.int8)
    last = {int(s): r for r, s in enumerate(slots.tolist())}
    at, of = torch.tensor(list(last)), torch.tensor(list(last.values()))
    assert torch.equal(codes.cpu()[at].double(), want[of]) and torch.equal(scales.cpu()[at], ws[of])


def test_empty_calls():
    codes, scales = kda.state_cache_empty(3, (2, 8), torch.int8, DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    kda.state_cache_write(torch.empty(0, 2, 8, device=DEV), codes, scales, none)
    assert kda.state_cache_read(codes, scales, none).shape == (0, 2, 8)
    codes, scales = kda.state_cache_empty(0, (2, 8), torch.int8, DEV)
    skip = torch.zeros(2, dtype=torch.int32, device=DEV)
    assert not kda.state_cache_read(codes, scales, skip).any()


def test_graph_and_stream():
    shape = (4, 64, 64)
    x = states_of(6, shape, 5).to(DEV)
    slots = torch.tensor([4, 1, 0, 7, 6, 2], dtype=torch.int32, device=DEV)
    codes, scales = kda.state_cache_empty(8, shape, torch.int8, DEV)
    want = kda.state_cache_read(*kda.state_cache_write(x, codes, scales, slots), slots)
    out = torch.empty_like(want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        kda.state_cache_read(codes, scales, slots, out=out)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.state_cache_write(x, codes, scales, slots)
        kda.state_cache_read(codes, scales, slots, out=out)
    for _ in range(3):
        codes.fill_(0), scales.fill_(0), out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        kda.state_cache_read(codes, scales)
