"""The 8-bit cache attention's ring of blocks, by its index arithmetic (no GPU needed): which lane copies a byte,
which lane reads it, and what stands between the reads of a place and the copies that refill it."""

from __future__ import annotations

import os
import re

import pytest

from exact_attention_63_gb300 import build

SOURCE = os.path.join(build.CSRC, "cache_attn_fp8.cu")


def run_at(d, r, c):
    return r * d + ((c ^ (r & 7) if d == 128 else c ^ ((r >> 1) & 3)) << 4)


def key_of(d, i):
    t = i >> 1
    return (2 * t + (t >> 1)) ^ ((i & 1) << 2) if d == 128 else i ^ (t & 1)


def copied(d):
    """Byte of a block's K (or V) -> the lane that copies it."""
    runs = d // 16
    step = 32 // runs
    out = {}
    for lane in range(32):
        for i in range(16 // step):
            at = run_at(d, lane // runs + i * step, lane % runs)
            for b in range(16):
                assert at + b not in out
                out[at + b] = lane
    return out


def read(d):
    """(lanes that read each byte of K, the same of V)."""
    k, v = {}, {}
    for lane in range(32):
        gr, t4 = lane >> 2, lane & 3
        for half in range(d // 64):
            for row in (key_of(d, gr), 8 + key_of(d, gr)):
                for b in range(16):
                    k.setdefault(run_at(d, row, 4 * half + t4) + b, set()).add(lane)
        for i in range(4):
            at = run_at(d, key_of(d, 2 * t4 + (i & 1)), gr if d == 128 else gr >> 1) + (0 if d == 128 else 8 * (gr & 1))
            for b in range(d // 8):
                v.setdefault(at + (i >> 1) * 8 * d + b, set()).add(lane)
    return k, v


@pytest.mark.parametrize("d", [64, 128])
def test_lanes_read_what_others_copy_so_the_warp_meets_before_a_place_is_refilled(d):
    copies = copied(d)
    assert sorted(copies) == list(range(16 * d))
    for reads in read(d):
        assert sorted(reads) == list(range(16 * d))  # every byte is read
        assert any(copies[at] not in lanes for at, lanes in reads.items())
    code = re.sub(r"//[^\n]*", "", open(SOURCE, encoding="utf-8").read())
    loop = code[code.index("copy_wait<L::kStages - 1>()"):code.index("st = st + 1 == L::kStages")]
    work, refill = loop.rindex("block(nv"), loop.index("copy(ahead, st)")
    # (inside `publish` the warp meets as well, but only before one copy in sixteen)
    between = re.sub(r"if \(phase == 0\) \{.*?\n      \}", "", loop[work:refill], flags=re.S)
    assert loop.index("__syncwarp()") < loop.index("block(16")
    assert "__syncwarp()" in between
