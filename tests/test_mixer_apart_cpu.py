"""States that the state space scan's single tokens update: refused on any other tensor of the call, by the C entry
points, also where they are updated in place (CPU; fake device addresses, never dereferenced)."""
import ctypes

import pytest

import kda_recurrent_state_amd as kda
from tests.test_mixer_boundary_cpu import ARGS, GOOD, INVALID, ssm
from tests.test_scan_launch_cpu import host_check

N, H, G, K, P, W = 3, 4, 2, 16, 8, 4
CH = H * P + 2 * G * K
BYTES = {"x": N * H * P * 2, "dt": N * H * 4, "A": H * 4, "B": N * G * K * 2, "C": N * G * K * 2, "D": H * 4, "dt_bias": H * 4,
         "h_in": N * H * K * P * 4, "h_out": N * H * K * P * 4, "y": N * H * P * 2, "xbc": N * CH * 2,
         "conv_weight": CH * W * 4, "conv_bias": CH * 4, "conv_state_in": N * (W - 1) * CH * 2,
         "conv_state_out": N * (W - 1) * CH * 2, "ws": N * CH * 4}
IN_PLACE = {"h_out": "h_in", "conv_state_out": "conv_state_in"}
CASES = [(fn, out, n, place) for fn, outs in (("kda_ssm_step", ["h_out"]), ("kda_ssm_conv_step", ["h_out", "conv_state_out"]))
         for out in outs for n in ARGS[fn][0].split() if n not in (out, IN_PLACE[out]) for place in (False, True)]


@pytest.mark.parametrize("fn,out,name,in_place", CASES, ids=str)
def test_a_state_on_another_tensor(fn, out, name, in_place):
    lib = kda.load_library()
    names = ARGS[fn][0].split()
    plain = (W, 1) if ARGS[fn][2] else ()
    for where in ("first byte", "last byte"):
        at = {n: GOOD + (i << 32) for i, n in enumerate(names)}
        if in_place:
            for o, i in IN_PLACE.items():
                if o in at:
                    at[o] = at[i]
        # all ends are multiples of 4 bytes (256 for the workspace, which stays where it is)
        moved, by = (out, name) if name in ("ws", "h_in", "conv_state_in", "h_out", "conv_state_out") else (name, out)
        at[moved] = at[by] - BYTES[moved] + 4 if where == "first byte" else at[by] + BYTES[by] - 4
        if in_place and moved in IN_PLACE:
            at[IN_PLACE[moved]] = at[moved]
        d = ssm(num_seqs=N, heads=H, total_tokens=N, groups=G, state=K, width=P)
        tail = ([ctypes.c_size_t(1 << 40)] if "ws" in names else []) + [None]
        status = getattr(lib, fn)(ctypes.byref(d), *plain, *[at[n] for n in names], *tail)
        message = lib.kda_last_error().decode()
        assert status == INVALID and "overlaps" in message, (where, status, message)


@pytest.mark.parametrize("fn,out", [("kda_ssm_step", "h_out"), ("kda_ssm_conv_step", "h_out"), ("kda_ssm_conv_step", "conv_state_out")])
def test_a_state_partly_on_itself(fn, out):
    lib = kda.load_library()
    names = ARGS[fn][0].split()
    for by in (4, -4, BYTES[out] - 4, 4 - BYTES[out]):
        at = {n: GOOD + (i << 32) for i, n in enumerate(names)}
        at[out] = at[IN_PLACE[out]] + by
        d = ssm(num_seqs=N, heads=H, total_tokens=N, groups=G, state=K, width=P)
        tail = ([ctypes.c_size_t(1 << 40)] if "ws" in names else []) + [None]
        plain = (W, 1) if ARGS[fn][2] else ()
        assert getattr(lib, fn)(ctypes.byref(d), *plain, *[at[n] for n in names], *tail) == INVALID
        assert "overlaps" in lib.kda_last_error().decode()


def test_extents_of_tokens_that_lie_apart(tmp_path):
    assert "extent check ok" in host_check("extent_check", tmp_path)
