"""The norms' reduction over lanes (csrc/norm.hip, lanes_reduce) leaves the same fp32 sum in every lane: its steps, as
the source has them, on numbers."""
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "quantized_grouped_gemm_token_amd", "csrc", "norm.hip")


def source_lane(ctrl, lane):
    """The lane that a DPP control reads for this one."""
    row, i = lane & ~15, lane & 15
    if ctrl < 0x100:                                         # a permutation of each quad
        return (lane & ~3) + (ctrl >> 2 * (lane & 3) & 3)
    if 0x121 <= ctrl <= 0x12F:                               # rows turned right
        return row + (i - (ctrl - 0x120)) % 16
    if ctrl == 0x140:                                        # rows mirrored
        return row + 15 - i
    if ctrl == 0x141:                                        # half rows mirrored
        return row + (i & 8) + 7 - (i & 7)
    raise AssertionError(f"unknown control {ctrl:#x}")


def steps():
    """(lanes a step is for, its controls) of lanes_reduce."""
    text = open(SOURCE).read()
    body = re.search(r"float lanes_reduce\(float v\) \{(.*?)\n\}", text, re.S).group(1)
    dpp = [(int(n), int(c, 16)) for n, c in
           re.findall(r"kLanes > (\d+)\) v = Op::of\(v, dpp<(0x[0-9A-Fa-f]+)>\(v\)\)", body)]
    swaps = [(int(n), int(k)) for n, k in
             re.findall(r"kLanes > (\d+)\) \{\s*const auto s = __builtin_amdgcn_permlane(\d+)_swap", body)]
    assert [n for n, _ in dpp] == [1, 2, 4, 8] and swaps == [(16, 16), (32, 32)]
    return dpp, swaps


def lanes_sum(v, lanes):
    """v fp32 [rows, 64] -> what each lane holds."""
    dpp, swaps = steps()
    for n, ctrl in dpp:
        if lanes > n:
            v = v + v[:, [source_lane(ctrl, lane) for lane in range(64)]]
    for n, width in swaps:                                   # the even and the odd of each pair of rows of `width`
        if lanes > n:
            even = [lane & ~width for lane in range(64)]
            v = v[:, even] + v[:, [lane | width for lane in even]]
    return v


@pytest.mark.parametrize("lanes", [2, 4, 8, 16, 64])
def test_every_lane_has_the_same_sum(lanes):
    rng = np.random.Generator(np.random.PCG64(lanes))
    # the sums of squares of lanes; fewer than 64 lanes hold theirs again and again, as the waves' sums are read
    parts = rng.chisquare(8, size=(20000, lanes)).astype(np.float32)
    got = lanes_sum(np.tile(parts, 64 // lanes), lanes)
    assert got.dtype == np.float32
    other = (got != got[:, :1]).any(1)
    assert not other.any(), f"{int(other.sum())} of {len(got)} rows have more than one sum"
    # log2(lanes) additions: half a step of each, of sums of positive numbers
    want = parts.astype(np.float64).sum(1)
    assert np.all(np.abs(got[:, 0] - want) <= 1.001 * np.log2(lanes) * 2.0 ** -24 * want)


@pytest.mark.parametrize("lanes", [2, 4, 8, 16, 64])
def test_every_lane_adds_each_value_once(lanes):
    parts = np.broadcast_to(np.arange(1, lanes + 1, dtype=np.float32) ** 2, (1, lanes))   # (exact in fp32)
    assert np.all(lanes_sum(np.tile(parts, 64 // lanes), lanes) == parts.sum())
