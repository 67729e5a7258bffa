"""The 8-bit cache's operators on the GPU against their float64 definitions."""

from __future__ import annotations

import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import cache_reference as ref
import fp8_cache_reference as ref8
from cache_reference import HALF_BF16, f64
from exact_attention_63_gb300 import attn, cache
from fp8_cache_reference import Fp8Case
from gpu_common import need_gpu
from test_cache_gpu import ATTEND

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    need_gpu()
    assert attn.get_status() == 0
    yield
    assert attn.get_status() == 0


def attend(c, **kw):
    return cache.attn_fwd_cache_fp8(c.q, c.k_new, c.v_new, *c.pages(), c.table, c.seq_lens, c.cu, c.max_new(),
                                    parents=c.parents, **kw)


def check(c, o, lse):
    O, L, A = ref.attention(c)
    # Scores: fp32 sums as for the bf16 cache; q's elements below 2^-28 of a row's largest are off by
    # less than 2^-39 of it, d of them by less than the sum's own rounding.
    eps = ref.score_bound(c)
    # P rounded to 16 bits (f16 for cached keys, bf16 for new ones: 2^-8 covers both) and, below
    # f16's range, by less than 2^-32 of the row's reference each; O rounded once.
    vmax = max([np.nan_to_num(np.abs(f64(x))).max(initial=0.0) for x in (c.v, c.v_new)])
    floor = (max(c.lens) + 128) * 2.0 ** -32 * vmax
    tol = HALF_BF16 * (A + np.abs(O)) * (1 + HALF_BF16) + (4 * eps + 2.0 ** -20) * A + floor
    err = np.abs(f64(o) - O)
    assert np.isfinite(f64(o)).all()
    assert (err <= tol).all(), f"O: {(err - tol).max():.3e} beyond its bound"
    tol_l = 2 * eps + 2.0 ** -20 * (1 + np.abs(L))
    err_l = np.abs(f64(lse) - L)
    assert (err_l <= tol_l).all(), f"LSE: {(err_l - tol_l).max():.3e} beyond its bound"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: c[0])
def test_attention(case, d):
    name, lens, new, H, hkv, page, tree = case
    c = Fp8Case(lens, new, H, hkv, d, page, seed=len(name), tree=tree).cuda()
    o, lse = attend(c)
    check(c, o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 2, 3, 9, 40])
def test_attention_of_blocks_of_different_scales(new, d):
    """Scales from 2^-12 to 2^12 times the usual: values of v in 2^24 sizes share one sum, and scores
    of hundreds move the reference."""
    c = Fp8Case([900, 333, 16, 31], [new, 1, new, 2], 8, 2, d, 32, seed=3, spread=12)
    c.scale = d ** -0.5 / 512
    c.cuda()
    o, lse = attend(c, scale=c.scale)
    check(c, o, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_extreme_scales(d):
    """Scale bytes at and beyond the ends of their range; q as small or large as makes the scores ordinary."""
    c = Fp8Case([200], [2], 4, 2, d, 16, seed=4)
    c.k_new.zero_()
    for byte, counts, size in ((10, 10, 2.0 ** 100), (0, 10, 2.0 ** 100), (246, 246, 2.0 ** -112), (255, 246, 2.0 ** -112)):
        x = Fp8Case([200], [2], 4, 2, d, 16, seed=4)
        x.k_new.zero_()
        x.k_scales.fill_(byte)
        x.k_codes[:] = torch.where(x.k_codes == 127, 127, x.k_codes & 0xBF)  # codes below 2: no score beyond hundreds
        k = ref8.values(x.k_codes.numpy(), np.full(x.k_scales.shape, counts, np.uint8))
        x.k = torch.from_numpy(k).bfloat16()
        x.q = (x.q.double() * size).bfloat16()
        x.scale = 2.0 ** 10 if counts == 10 else 2.0 ** -10
        O, L, A = ref.attention(x)
        x.cuda()
        o, lse = attend(x, scale=x.scale)
        assert np.isfinite(O).all() and np.isfinite(f64(o)).all()
        big = np.abs(f64(x.q)).max() * np.nan_to_num(np.abs(k)).max() * d * x.scale
        eps = (d + 8) * ref.HALF_F32 * big + 2.0 ** -20
        assert (np.abs(f64(o) - O) <= HALF_BF16 * (A + np.abs(O)) * (1 + HALF_BF16) + (4 * eps + 2.0 ** -20) * A + 1e-6).all()
        assert (np.abs(f64(lse) - L) <= 2 * eps + 2.0 ** -20 * (1 + np.abs(L))).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sigma", [6.0, 1e-30, 1e30])
def test_attention_of_small_and_large_queries(sigma, d):
    c = Fp8Case([700, 90], [3, 20], 8, 2, d, 32, seed=5, sigma=sigma)
    c.scale = d ** -0.5 * (1.0 if sigma == 6.0 else 1.0 / sigma)
    if sigma != 6.0:
        c.k_new.mul_(0.5)
    c.cuda()
    o, lse = attend(c, scale=c.scale)
    check(c, o, lse)


def test_attention_of_queries_of_many_sizes():
    """A row whose elements span 2^30: the small ones meet large keys."""
    c = Fp8Case([300], [2], 4, 2, 128, 16, seed=6)
    c.q *= (2.0 ** -torch.arange(128).remainder(31).float()).bfloat16()
    c.cuda()
    o, lse = attend(c)
    check(c, o, lse)


def test_attention_growing_scores():
    """Every key scores higher than the ones before."""
    c = Fp8Case([1200], [2], 4, 2, 128, 16, seed=7, tree="chain")
    j = torch.arange(1200)
    rows = c.table[0, j // 16].long(), j % 16
    x = (j / 100.0)[:, None, None].expand(1200, 2, 128).double().numpy()
    codes, scales = c.k_codes.numpy(), c.k_scales.numpy()
    ref8.append(codes, scales, c.table.numpy(), [1200], [0, 1200], x)
    c.k = torch.from_numpy(ref8.values(codes, scales)).bfloat16()
    c.q[:] = 1.0
    c.k_new[:] = 13.0
    assert torch.isfinite(c.k[rows].float()).all()
    c.cuda()
    o, lse = attend(c)
    check(c, o, lse)


def test_attention_leaves_other_rows_alone():
    c = Fp8Case([100, 260], [2, 3], 4, 2, 64, 16, seed=7)
    pad = 6
    for name in ("q", "k_new", "v_new"):
        t = getattr(c, name)
        setattr(c, name, torch.cat([t, torch.full((pad,) + t.shape[1:], float("nan")).bfloat16()]))
    c.parents = torch.cat([c.parents, torch.full((pad,), 99, dtype=torch.int32)])
    total, c.total = c.total, c.total + pad
    c.cuda()
    out = torch.full((c.total, 4, 64), 7.0, device="cuda").bfloat16()
    lse = torch.full((4, c.total), 7.0, device="cuda")
    attend(c, out=out, lse=lse)
    c.total = total
    for name in ("q", "k_new", "v_new", "parents"):
        setattr(c, name, getattr(c, name)[:total])
    check(c, out[:total], lse[:, :total])
    assert (out[total:] == 7).all() and (lse[:, total:] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_of_nan_in_a_live_key(new, d):
    """A NaN code in a sequence's keys or values reaches its own rows and no other sequence's or head's."""
    c = Fp8Case([300, 300], [new, new], 4, 2, d, 16, seed=9).cuda()
    good, good_lse = attend(c)
    c.k_codes[c.table[0, 3].long(), 5, 1] = 127
    c.v_codes[c.table[1, 2].long(), 1, 0, 7] = 255
    o, lse = attend(c)
    r0, r1 = slice(0, new), slice(new, 2 * new)
    assert o[r0, 2:].isnan().all() and lse[2:, r0].isnan().all()
    assert torch.equal(o[r0, :2], good[r0, :2]) and torch.equal(o[r1, 2:], good[r1, 2:])
    assert o[r1, :2, 7].isnan().all() and torch.equal(lse[:, r1], good_lse[:, r1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 33])
def test_attention_of_strided_views_streams_and_graphs(new, d):
    """Pages stored head by head, q, k and v as slices of one projection, typed codes; on another
    stream; captured, and replayed with other lengths and contents: all give the same bits."""
    c = Fp8Case([500, 37, 129], [new, new, 1], 8, 2, d, 32, seed=10, room=100).cuda()
    o, lse = attend(c)
    check(c, o, lse)
    packed = torch.cat([c.q, c.k_new, c.v_new], 1)
    q, kn, vn = packed[:, :8], packed[:, 8:10], packed[:, 10:]
    k, v = (x.transpose(1, 2).contiguous().transpose(1, 2).view(torch.float8_e4m3fn) for x in (c.k_codes, c.v_codes))
    ks, vs = c.k_scales.view(torch.float8_e8m0fnu), c.v_scales.view(torch.float8_e8m0fnu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = cache.attn_fwd_cache_fp8(q, kn, vn, k, v, ks, vs, c.table, c.seq_lens, c.cu, new, parents=c.parents, stream=side)
    side.synchronize()
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    ws = torch.empty(cache.workspace_size_fp8(8, 2, 128, d), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = attend(c, workspace=ws)
    graph.replay()
    assert torch.equal(o3, o) and torch.equal(lse3, lse)
    c.seq_lens.copy_(torch.tensor([20, 37, 1]))
    c.lens = [20, 37, 1]
    graph.replay()
    check(c, o3, lse3)


def test_attention_repeats_bit_for_bit():
    g = torch.Generator().manual_seed(23)
    n = 100
    lens = [int(x) for x in torch.randint(0, 900, (n,), generator=g)]
    new = [40 if x else 3 for x in torch.randint(0, 2, (n,), generator=g).tolist()]
    for d in (64, 128):
        c = Fp8Case(lens, new, 8, 2, d, 16, seed=24).cuda()
        o, lse = attend(c)
        check(c, o, lse)
        for _ in range(50):
            o2, lse2 = attend(c)
            assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_options_of_a_kernel_that_waits_for_nobody():
    """Few rows: no warp waits for copies of another, so there is nothing to withhold and no limit to reach."""
    c = Fp8Case([300, 77], [2, 1], 8, 2, 128, 16, seed=11).cuda()
    o, lse = attend(c, options=attn.make_options(timeout_ms=20, test_flags=attn.TEST_WITHHOLD_KV))
    check(c, o, lse)
    o, lse = attend(c)
    check(c, o, lse)


def test_malformed_tables_stay_inside():
    """Pages, lengths and offsets out of range: no fault, no write outside the outputs."""
    c = Fp8Case([300, 90, 40], [3, 2, 1], 4, 2, 64, 16, seed=12).cuda()
    guard = torch.full((c.total + 8, 4, 64), 3.0, device="cuda").bfloat16()
    lse = torch.empty((4, c.total), device="cuda")
    c.table[0, 3], c.table[1, 0] = 1 << 30, -5
    c.seq_lens.copy_(torch.tensor([1 << 30, -7, 40]))
    attend(c, out=guard[4:-4], lse=lse)
    assert (guard[:4] == 3).all() and (guard[-4:] == 3).all()
    k, v = c.k_codes.clone(), c.v_codes.clone()
    cache.cache_append_fp8(c.k_new, c.v_new, *c.pages(), c.table, c.seq_lens, c.cu)
    cache.cache_gather_fp8(*c.pages(), c.table, c.seq_lens, c.cu, c.total)
    torch.cuda.synchronize()
    assert k.shape == c.k_codes.shape and v.shape == c.v_codes.shape


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,group,new", [(8, 4, 1), (8, 1, 8), (6, 2, 1), (16, 1, 1), (16, 3, 4), (12, 2, 5), (5, 4, 4), (8, 4, 8), (8, 8, 5),
                                           (2, 40, 1), (1, 33, 1), (1, 16, 1), (4, 17, 1), (8, 4, 33)])
def test_attention_of_head_counts(hkv, group, new, d):
    """Runs of 8, 4, 2 and 1 key heads, tiles of 8, 16, 32 and more rows, one sequence and several."""
    for lens in ([300], [129, 0, 700, 33]):
        c = Fp8Case(lens, [new, 1, new, 0][:len(lens)], hkv * group, hkv, d, 48, seed=hkv).cuda()
        o, lse = attend(c)
        check(c, o, lse)


@pytest.mark.parametrize("new", [1, 3, 9, 40])
def test_attention_of_2048_sequences(new):
    """The most sequences of a call: their table is as large as it gets beside every kernel's tiles."""
    lens = [(7 * i) % 40 for i in range(2048)]
    c = Fp8Case(lens, [new if i % 97 == 0 else int(i % 5 == 0) for i in range(2048)], 4, 1, 64, 16, seed=19).cuda()
    o, lse = attend(c)
    check(c, o, lse)


@pytest.mark.parametrize("n_seq,hkv,group,new,d", [(700, 8, 4, 1, 128), (2048, 8, 2, 2, 128), (1900, 8, 1, 3, 64), (1300, 2, 4, 2, 64), (1250, 3, 8, 1, 128),
                                                   (640, 16, 2, 1, 128), (420, 8, 4, 6, 128), (330, 8, 4, 8, 64), (400, 4, 8, 20, 64)])
def test_attention_of_many_tiles(n_seq, hkv, group, new, d):
    """More tiles than CTAs, by far: ranges of each group of warps, and a join that goes by the ranges' ends."""
    lens = [(37 * i * i + 11) % 70 if i % 9 else 0 for i in range(n_seq)]
    news = [new if i % 3 else (i // 3) % (new + 1) for i in range(n_seq)]
    c = Fp8Case(lens, news, hkv * group, hkv, d, 32, seed=n_seq).cuda()
    o, lse = attend(c)
    check(c, o, lse)


def test_random_calls():
    """Seeded calls over the range of the contract: heads, groups, pages, lengths from 0, trees, padded bounds."""
    r = np.random.default_rng(20)
    for i in range(60):
        n, hkv = int(r.integers(1, 9)), int(r.choice([1, 2, 3, 4, 8]))
        group, d, page = int(r.choice([1, 2, 3, 4, 7, 8])), int(r.choice([64, 128])), int(r.choice([16, 32, 48, 64, 128, 256]))
        new = [int(x) for x in r.choice([0, 1, 1, 2, 4, 7, 13, 40, 128], n)]
        lens = [int(x) for x in r.integers(0, int(r.choice([20, 300, 1500])), n)]
        if not sum(new):
            new[0] = 1
        c = Fp8Case(lens, new, hkv * group, hkv, d, page, seed=i, tree=str(r.choice(["random", "chain", "roots", "line"])),
                    spread=int(r.choice([0, 0, 3]))).cuda()
        o, lse = cache.attn_fwd_cache_fp8(c.q, c.k_new, c.v_new, *c.pages(), c.table, c.seq_lens, c.cu,
                                          min(128, c.max_new() + int(r.choice([0, 0, 5]))), parents=c.parents)
        check(c, o, lse)


def test_first_calls_in_a_graph_and_from_two_threads():
    """A process whose first calls are captured, and two threads with streams of their own."""
    code = textwrap.dedent("""
        import sys
        sys.path[:0] = ["tests", "."]
        import torch
        from concurrent.futures import ThreadPoolExecutor
        from exact_attention_63_gb300 import attn, cache, rotary
        from fp8_cache_reference import Fp8Case
        from test_cache_fp8_gpu import attend, check
        cases = [Fp8Case([200, 33], [t, 1], 8, 2, 128, 16, seed=t).cuda() for t in (1, 40)]
        freq = rotary.rotary_frequencies(128).cuda()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [attend(c) for c in cases]
            turned = rotary.rotary_fwd(cases[0].q, cases[0].k_new, None, freq)
            lens = cases[0].seq_lens
            cache.cache_gather_fp8(*cases[0].pages(), cases[0].table, lens, cases[0].cu, cases[0].total)
        graph.replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            check(c, *o)
        def work(i):
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    o = attend(cases[i])
                torch.cuda.current_stream().synchronize()
                return o
        with ThreadPoolExecutor(2) as pool:
            for o, want in zip(pool.map(work, (0, 1)), outs):
                assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
        assert attn.get_status() == 0
    """)
    subprocess.run([sys.executable, "-c", code], check=True, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), timeout=240)


@pytest.mark.parametrize("d", [64, 128])
def test_wait_limit(d):
    """Many rows: the converters lay out no keys, the call ends, the status says so, and the next call is right."""
    c = Fp8Case([300, 77], [40, 1], 8, 2, d, 16, seed=11).cuda()
    attend(c, options=attn.make_options(timeout_ms=20, test_flags=attn.TEST_WITHHOLD_KV))
    assert attn.get_status() == -8
    o, lse = attend(c)
    check(c, o, lse)


# ------------------------------------------------------------------ append and gather

APPEND = [
    ("one", [1], [1], 16), ("fills", [16, 17, 31, 32, 33], [16, 1, 15, 16, 2], 16), ("joins", [5, 20, 47, 100], [2, 3, 16, 37], 32),
    ("whole", [300, 129, 1], [300, 129, 1], 48), ("none", [40, 7, 0, 90], [0, 7, 0, 1], 16), ("steps", [(17 * i) % 90 + 1 for i in range(70)], [1] * 70, 64),
    ("too_many", [3, 40], [20, 41], 16),
]


def put(c, rows=None, cu=None, lens=None):
    """The append on the GPU and by definition; the codes and scales have to agree bit for bit."""
    want = []
    table = c.table.cpu().numpy()
    for name in ("k", "v"):
        codes, scales = getattr(c, name + "_codes").cpu().numpy().copy(), getattr(c, name + "_scales").cpu().numpy().copy()
        ref8.append(codes, scales, table, lens, cu, f64(getattr(c, name + "_new")), rows)
        want.append((codes, scales))
    rows = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    cache.cache_append_fp8(c.k_new, c.v_new, *c.pages(), c.table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           torch.tensor(cu, dtype=torch.int32, device="cuda"), rows=rows)
    for name, (codes, scales) in zip(("k", "v"), want):
        assert np.array_equal(getattr(c, name + "_scales").cpu().numpy(), scales), name
        assert np.array_equal(getattr(c, name + "_codes").cpu().numpy(), codes), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: c[0])
def test_append(case, d):
    """Sizes of 2^-3 to 2^3 times the cache's: scales that grow, stay, and are new."""
    name, lens, new, page = case
    before = [max(a - t, 0) for a, t in zip(lens, new)]
    c = Fp8Case(before, new, 6, 3, d, page, seed=len(name), room=max(new) + 1)
    g = torch.Generator().manual_seed(len(name))
    for x in (c.k_new, c.v_new):
        x *= torch.exp2(torch.randint(-3, 4, (c.total, 3, 1), generator=g).float()).bfloat16()
    c.cuda()
    put(c, cu=c.cu.tolist(), lens=lens)


@pytest.mark.parametrize("d", [64, 128])
def test_append_of_special_values(d):
    """Infinities, NaN, zeros, the smallest and largest numbers, ties between codes."""
    special = [0.0, -0.0, float("inf"), float("-inf"), float("nan"), 2.0 ** -133, -(2.0 ** -126), 3.3895e38, -3.3895e38,
               448.0, 449.0, 464.0, 466.0, 480.0, 1.0625, 1.1875, -2.125, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11]
    c = Fp8Case([20, 3], [len(special) + 12, 40], 2, 2, d, 32, seed=2, room=100)
    for i, x in enumerate(special):
        c.k_new[i, 0, i % d] = x                 # in blocks of ordinary numbers
        c.k_new[i, 1, :] = x                     # a row of it
        c.v_new[i, :, :] = x if abs(x) <= 480 else 0.0
    c.v_new[len(special):] = 0.0                 # blocks of zeros
    c.k_new[len(special):, 1] = float("inf")     # blocks without a finite value
    c.cuda()
    put(c, cu=c.cu.tolist(), lens=[20 + len(special) + 12, 43])


def test_append_rounds_every_tie_as_the_definition_does():
    """All bf16 numbers between the codes' neighbours from 2^-12 to 512, in blocks of scale 1."""
    bits = torch.arange(0x3980, 0x4400, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[bits <= 448]
    n = -(-len(bits) // 15)
    rows = torch.zeros(16 * n, 1, 64).bfloat16()
    rows[::16] = 448.0  # each block's scale is 1
    for i in range(n):
        part = bits[15 * i:15 * i + 15]
        rows[16 * i + 1:16 * i + 1 + len(part), 0, 3] = part
        rows[16 * i + 1:16 * i + 1 + len(part), 0, 40] = -part
    c = Fp8Case([0], [16 * n], 1, 1, 64, 16, seed=2, room=16 * n)
    c.k_new, c.v_new = rows, rows.clone()
    c.cuda()
    put(c, cu=[0, 16 * n], lens=[16 * n])


def test_append_of_accepted_rows():
    c = Fp8Case([30, 50, 16], [8, 8, 8], 4, 2, 128, 16, seed=13, room=20).cuda()
    put(c, rows=[0, 3, 7, 8, -1, 24, 15, 16, 16], cu=[0, 3, 7, 9], lens=[33, 54, 18])


def test_append_token_by_token_is_append_of_all_where_scales_do_not_grow():
    """A block's codes depend on when its largest value came only by the rounding to larger scales:
    with the largest value first there is none."""
    a, b = (Fp8Case([0], [40], 2, 2, 64, 16, seed=14, room=48).cuda() for _ in range(2))
    for c in (a, b):
        c.k_new[::16], c.v_new[::16] = 9.0, -9.0
    cache.cache_append_fp8(a.k_new, a.v_new, *a.pages(), a.table, torch.tensor([40], dtype=torch.int32, device="cuda"), a.cu)
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(40):
        cache.cache_append_fp8(b.k_new[i:i + 1], b.v_new[i:i + 1], *b.pages(), b.table,
                               torch.tensor([i + 1], dtype=torch.int32, device="cuda"), one)
    for x, y in zip(a.pages(), b.pages()):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
def test_append_and_gather_of_strided_views(d):
    c = Fp8Case([40, 20], [5, 30], 4, 2, d, 32, seed=15, room=40)
    c2 = Fp8Case([40, 20], [5, 30], 4, 2, d, 32, seed=15, room=40)
    c.cuda(), c2.cuda()
    lens = torch.tensor([45, 50], dtype=torch.int32, device="cuda")
    cache.cache_append_fp8(c.k_new, c.v_new, *c.pages(), c.table, lens, c.cu)
    both = torch.cat([c2.k_new, c2.v_new], 1)
    k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (c2.k_codes, c2.v_codes))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.cache_append_fp8(both[:, :2], both[:, 2:], k, v, c2.k_scales, c2.v_scales, c2.table, lens, c2.cu, stream=side)
    cu = torch.tensor([0, 45, 95], dtype=torch.int32, device="cuda")
    got = cache.cache_gather_fp8(k, v, c2.k_scales, c2.v_scales, c2.table, lens, cu, 95, stream=side)
    side.synchronize()
    want = cache.cache_gather_fp8(*c.pages(), c.table, lens, cu, 95)
    assert torch.equal(k, c.k_codes) and torch.equal(v, c.v_codes) and torch.equal(c.k_scales, c2.k_scales)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,hkv", [(16, 1), (48, 3), (128, 8)])
def test_gather(page, hkv, d):
    lens = [1, 16, 0, 47, 300]
    c = Fp8Case(lens, [1] * 5, hkv, hkv, d, page, seed=16, spread=30).cuda()
    for n in (lens, [1, 3, 0, 47, 129], [0, 0, 0, 0, 0], [2, 16, 5, 40, 300]):
        cu = torch.tensor([0] + np.cumsum(n).tolist(), dtype=torch.int32, device="cuda")
        total = int(cu[-1]) + 4
        k, v = (torch.full((total, hkv, d), 5.0, device="cuda").bfloat16() for _ in range(2))
        cache.cache_gather_fp8(*c.pages(), c.table, c.seq_lens, cu, total, k, v)
        for got, x in ((k, c.k), (v, c.v)):
            want = torch.full_like(got, 5.0)
            for s, m in enumerate(n):
                for i in range(max(0, m - lens[s]), m):
                    j = lens[s] - m + i
                    want[int(cu[s]) + i] = x[int(c.table[s, j // page]), j % page]
            assert torch.equal(got, want)


def test_offsets_beyond_32_bits():
    """A page that lies beyond 2^32 bytes."""
    n_pages, page, hkv, d = 4200, 1024, 8, 128  # 4.4 GB of codes
    k = torch.zeros((n_pages, page, hkv, d), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.zeros((n_pages, hkv, page // 16), dtype=torch.uint8, device="cuda")
    vs = torch.zeros_like(ks)
    c = Fp8Case([0], [40], 8, 8, d, 16, seed=17, tree="chain", room=48).cuda()
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    cache.cache_append_fp8(c.k_new, c.v_new, k, v, ks, vs, table, lens, c.cu)
    got = cache.cache_gather_fp8(k, v, ks, vs, table, lens, c.cu, 40)
    cache.cache_append_fp8(c.k_new, c.v_new, *c.pages(), c.table, lens, c.cu)
    want = cache.cache_gather_fp8(*c.pages(), c.table, lens, c.cu, 40)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    x = (c.q[:1], c.k_new[:1], c.v_new[:1])
    far = cache.attn_fwd_cache_fp8(*x, k, v, ks, vs, table, lens, one, 1)
    near = cache.attn_fwd_cache_fp8(*x, *c.pages(), c.table, lens, one, 1)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])


def test_empty_calls():
    c = Fp8Case([30], [0], 4, 2, 64, 16, seed=18).cuda()
    o, lse = cache.attn_fwd_cache_fp8(c.q, c.k_new, c.v_new, *c.pages(), c.table, c.seq_lens, c.cu, 1)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    cache.cache_append_fp8(c.k_new, c.v_new, *c.pages(), c.table, c.seq_lens, c.cu)
    k, v = cache.cache_gather_fp8(*c.pages(), c.table, c.seq_lens, c.cu, 0)
    assert k.shape == v.shape == (0, 2, 64)
