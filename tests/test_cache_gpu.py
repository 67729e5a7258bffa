"""The cache operators on the GPU against their float64 definitions."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import cache_reference as ref
from cache_reference import HALF_BF16, HALF_F32, Case, f64
from exact_attention_63_gb300 import attn, cache
from gpu_common import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    need_gpu()
    assert attn.get_status() == 0
    yield
    assert attn.get_status() == 0


def attend(c: Case, **kw):
    return cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, c.max_new(),
                                parents=c.parents, **kw)


def check_attention(c: Case, o, lse, rows=slice(None)):
    O, L, A = ref.attention(c)
    eps = ref.score_bound(c)
    # P rounded once (2^-8 of each p|v|), O rounded once, scores off by eps each
    # (numerator and sum), 2^-20 for the exponentials and the fp32 sums.
    tol = HALF_BF16 * (A + np.abs(O)) * (1 + HALF_BF16) + (4 * eps + 2.0 ** -20) * A
    err = np.abs(f64(o) - O)
    assert np.isfinite(f64(o)[rows]).all()
    assert (err <= tol)[rows].all(), f"O: {(err - tol).max():.3e} beyond its bound"
    tol_l = 2 * eps + 2.0 ** -20 * (1 + np.abs(L))
    err_l = np.abs(f64(lse) - L)
    assert (err_l <= tol_l)[:, rows].all(), f"LSE: {(err_l - tol_l).max():.3e} beyond its bound"


# lens, new tokens, H, H_kv, page, tree
ATTEND = [
    ("one", [1000], [1], 8, 2, 16, "chain"),
    ("empty_cache", [0, 0], [1, 5], 4, 4, 16, "random"),
    ("edges", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257], [1, 2, 1, 3, 1, 1, 1, 2, 1, 128, 1], 4, 2, 32, "random"),
    ("some_none", [40, 300, 5, 130], [0, 3, 0, 1], 6, 2, 48, "random"),
    ("tails", [112, 113, 64, 65, 100, 120], [16, 16, 64, 64, 17, 8], 2, 1, 16, "random"),
    ("big_pages", [500, 1], [4, 4], 4, 1, 256, "random"),
    ("page64", [190, 192, 70], [60, 64, 64], 4, 2, 64, "random"),
    ("wide_group", [333], [5], 128, 1, 16, "random"),
    ("group7", [400, 77], [33, 19], 14, 2, 16, "random"),
    ("deep", [130, 260], [128, 127], 4, 4, 128, "line"),
    ("chain128", [130, 260], [128, 100], 4, 4, 128, "chain"),
    ("roots", [9, 250], [40, 128], 6, 3, 16, "roots"),
    ("long", [20011], [2], 4, 1, 128, "random"),
    ("long_wide", [9000, 130], [80, 3], 8, 1, 64, "random"),
    ("long_pair", [12000], [33], 8, 2, 16, "random"),
    ("one_or_two_tiles", [(53 * i) % 700 for i in range(120)], [40 if i % 3 == 1 else 1 + i % 4 for i in range(120)], 8,
     2, 16, "random"),
    ("many", [(37 * i) % 301 for i in range(333)], [1 + (i % 3 == 0) for i in range(333)], 2, 1, 16, "random"),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: c[0])
def test_attention(case, d):
    name, lens, new, H, hkv, page, tree = case
    c = Case(lens, new, H, hkv, d, page, seed=len(name), tree=tree).cuda()
    o, lse = attend(c)
    check_attention(c, o, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_one_row_tile_and_two_in_turn(d):
    """Runs of blocks without rows for the second tile, between blocks that have some and
    end in a tail (whose unused rows of V are zeroed): launches with their own timing."""
    g = torch.Generator().manual_seed(23)
    n = 150
    lens = [int(x) for x in torch.randint(0, 900, (n,), generator=g)]
    new = [40 if x else 3 for x in torch.randint(0, 2, (n,), generator=g).tolist()]
    c = Case(lens, new, 8, 2, d, 16, seed=24).cuda()
    o, lse = attend(c)
    check_attention(c, o, lse)
    for _ in range(200):
        o2, lse2 = attend(c)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_peaky_scores(d):
    """Standard deviation 6 in q: the reference maximum moves between blocks."""
    c = Case([1500, 700], [3, 20], 8, 2, d, 32, seed=5, sigma=6.0).cuda()
    o, lse = attend(c)
    check_attention(c, o, lse)


def test_attention_growing_scores():
    """Every key scores higher than the ones before: each block rescales."""
    c = Case([1200], [2], 4, 2, 128, 16, seed=6, tree="chain")
    u = torch.ones(128).bfloat16()
    c.q[:] = u
    for j in range(1200):
        c.k[int(c.table[0, j // 16]), j % 16] = (u.float() * (j / 100.0)).bfloat16()
    c.k_new[:] = (u.float() * 13).bfloat16()
    c.cuda()
    o, lse = attend(c)
    check_attention(c, o, lse)


def test_attention_leaves_other_rows_alone():
    """Rows behind the last sequence, and slots nobody uses, stay as they were."""
    c = Case([100, 260], [2, 3], 4, 2, 64, 16, seed=7)
    pad = 6
    for name in ("q", "k_new", "v_new"):
        t = getattr(c, name)
        setattr(c, name, torch.cat([t, torch.full((pad,) + t.shape[1:], float("nan")).bfloat16()]))
    c.parents = torch.cat([c.parents, torch.full((pad,), 99, dtype=torch.int32)])
    total = c.total + pad
    c.cuda()
    o = torch.full((total, 4, 64), 7.0, device="cuda").bfloat16()
    lse = torch.full((4, total), 7.0, device="cuda")
    k0, v0 = c.k.clone(), c.v.clone()
    attend(c, out=o, lse=lse)
    assert (o[c.total:] == 7).all() and (lse[:, c.total:] == 7).all()
    assert torch.equal(k0.view(torch.int16), c.k.view(torch.int16))
    assert torch.equal(v0.view(torch.int16), c.v.view(torch.int16))
    c.total, c.q, c.k_new, c.v_new, c.parents = total - pad, c.q[:-pad], c.k_new[:-pad], c.v_new[:-pad], c.parents[:-pad]
    check_attention(c, o[:-pad], lse[:, :-pad])


def test_attention_bad_parents_are_roots():
    c = Case([50], [4], 2, 1, 64, 16, seed=8)
    c.parents = torch.tensor([5, 1, -9, 1], dtype=torch.int32)  # 5 > 0, 1 = itself, -9, 1 (fine)
    good = Case([50], [4], 2, 1, 64, 16, seed=8)
    good.parents = torch.tensor([-1, -1, -1, 1], dtype=torch.int32)
    a, b = attend(c.cuda()), attend(good.cuda())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_attention(good, *b)


def test_attention_malformed_tables_stay_inside():
    """Lengths, pages and offsets outside their ranges: clamped, no access outside."""
    c = Case([100, 64], [2, 2], 2, 1, 64, 16, seed=9).cuda()
    c.table[:] = torch.tensor([-5, 1 << 30, 3, 2, 1, 0, 99], dtype=torch.int32, device="cuda")
    c.seq_lens[:] = torch.tensor([1 << 30, -4], dtype=torch.int32, device="cuda")
    c.cu[:] = torch.tensor([-3, 2, 900], dtype=torch.int32, device="cuda")
    attend(c)
    torch.cuda.synchronize()


def test_attention_strided_inputs_and_head_major_pages():
    """q, k_new, v_new as slices of one packed projection; pages stored head by head."""
    H, hkv, d = 8, 2, 128
    c = Case([300, 31], [3, 1], H, hkv, d, 32, seed=10)
    packed = torch.cat([c.q, c.k_new, c.v_new], 1).cuda()
    c.cuda()
    want = attend(c)
    c.q, c.k_new, c.v_new = packed[:, :H], packed[:, H:H + hkv], packed[:, H + hkv:]
    c.k = c.k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    both = torch.stack([c.v, c.v], 0)
    c.v = both[1]
    got = attend(c)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    check_attention(c, *got)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), torch.finfo(torch.bfloat16).min])
def test_attention_ignores_what_unused_slots_hold(value):
    c = Case([77, 200], [2, 4], 4, 2, 64, 16, seed=11)
    for t in (c.k, c.v):
        t[torch.isnan(t)] = value
    c.cuda()
    check_attention(c, *attend(c))


def test_attention_repeats_bit_for_bit():
    c = Case([4000, 9, 700], [5, 1, 60], 8, 2, 128, 32, seed=12).cuda()
    a = attend(c)
    for _ in range(20):
        b = attend(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_wait_limit():
    """Withheld copies: the wait runs out, the status says so, the next call is right."""
    c = Case([300], [2], 4, 2, 64, 16, seed=13).cuda()
    attend(c, options=attn.make_options(timeout_ms=50, test_flags=attn.TEST_WITHHOLD_KV))
    assert attn.get_status() == -8
    check_attention(c, *attend(c))


@pytest.mark.parametrize("which", ["attend", "weigh"])
def test_wait_limit_with_two_tiles(which):
    """The other kernels' waits run out as cleanly."""
    c = Case([3000, 40], [60, 1], 8, 2, 128, 16, seed=14).cuda()
    opts = attn.make_options(timeout_ms=50, test_flags=attn.TEST_WITHHOLD_KV)
    lse = torch.full((8, c.total), 6.0, device="cuda")
    start = f64(c.weights)
    if which == "attend":
        attend(c, options=opts)
    else:
        weigh(c, lse, out=torch.zeros_like(c.weights), options=opts)
    assert attn.get_status() == -8
    check_attention(c, *attend(c))
    check_weights(c, lse, start, weigh(c, lse))


# ------------------------------------------------------------------ weights
def weigh(c: Case, lse, **kw):
    return cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, c.max_new(), c.weights, **kw)


def check_weights(c: Case, lse, start, out):
    W = ref.weights(c, lse, start)
    base = ref.weights(c, lse, None)
    used = ~np.isnan(W)
    n_terms = max(c.new) * (c.H // c.hkv)
    eps = ref.score_bound(c)
    # each exponential: its score off by eps, its argument rounded (|argument| < 64
    # wherever the term counts), 2^-21 for the base-2 exponential; then the fp32 sum.
    rel = 2 * eps + 64 * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -24 * (n_terms / 32 + 64)
    tol = rel * np.abs(base) + HALF_F32 * 2 * np.abs(W) + 1e-30
    got = f64(out)
    assert np.isfinite(got[used]).all()
    err = np.abs(got - W)
    assert (err[used] <= tol[used]).all(), f"{(err - tol)[used].max():.3e} beyond its bound"


# lens, queries, H, H_kv, page
WEIGH = [
    ("one", [1000], [1], 8, 2, 16),
    ("edges", [1, 15, 16, 127, 128, 129, 255, 256, 257, 511, 513], [1, 1, 2, 3, 1, 1, 1, 2, 1, 8, 1], 4, 2, 32),
    ("some_none", [40, 300, 5, 130, 0], [0, 3, 0, 1, 0], 6, 2, 48),
    ("prompt", [700], [700], 4, 2, 64),
    ("prompts", [300, 5, 129, 600], [300, 5, 129, 600], 6, 1, 16),
    ("window", [900, 1300], [64, 64], 14, 2, 128),
    ("second_part", [900], [513], 2, 2, 256),
    ("wide_group", [333], [3], 128, 1, 16),
    ("more_queries_than_keys", [5, 20], [9, 20], 2, 1, 16),
    ("many", [1 + (37 * i) % 301 for i in range(333)], [1 for i in range(333)], 2, 1, 16),
    ("many_prompts", [1 + (97 * i) % 400 for i in range(40)], [1 + (97 * i) % 400 for i in range(40)], 4, 2, 16),
    ("prompt_and_steps", [1500, 3, 700, 256], [1500, 1, 0, 2], 4, 1, 64),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", WEIGH, ids=lambda c: c[0])
def test_weights(case, d):
    name, lens, new, H, hkv, page = case
    c = Case(lens, new, H, hkv, d, page, seed=len(name)).cuda()
    start = f64(c.weights)
    # any LSE will do; near the true one, with rows that add nothing among them
    lse = (torch.randn((H, c.total), generator=torch.Generator().manual_seed(1)) * 0.1 +
           float(np.log(np.mean(lens) + 1))).cuda()
    lse[0, 0] = -float("inf")
    lse[-1, -1] = float("inf")
    other = torch.full_like(c.weights, 5.0)
    assert weigh(c, lse, out=other) is other
    check_weights(c, lse, start, other)
    unused = torch.isnan(c.weights)
    assert (other[unused] == 5).all()
    assert weigh(c, lse) is c.weights
    assert torch.equal(c.weights[~unused], other[~unused]) and torch.isnan(c.weights[unused]).all()
    fresh = torch.zeros_like(c.weights)
    cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, c.max_new(), out=fresh)
    check_weights(c, lse, np.zeros_like(start), fresh)


def test_weights_of_every_query_sum_to_its_heads():
    """With the true LSE each (query, head) hands out weight 1 in all."""
    c = Case([513, 40], [513, 40], 8, 2, 128, 32, seed=3).cuda()
    c.weights.zero_()
    lse = torch.zeros(8, c.total)
    q, k = f64(c.q), f64(c.k)
    for s in range(2):
        r = slice(int(c.cu[s]), int(c.cu[s + 1]))
        K = ref.rows_of(k, c.table.cpu(), s, c.lens[s])
        for h in range(8):
            z = q[r, h] @ K[:, h // 4].T * c.scale
            z[np.triu_indices(len(z), 1)] = -np.inf
            lse[h, r] = torch.from_numpy(np.log(np.exp(z).sum(1)))
    out = weigh(c, lse.cuda())
    assert abs(float(out.double().sum()) - 8 * c.total) < 1e-5 * 8 * c.total


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prompt", [False, True])
def test_weights_of_short_and_long_tiles_in_turn(d, prompt):
    """Tiles of one half and of two follow each other on every CTA in any order, many
    of them and each launch with its own timing: the halves run apart and meet again."""
    g = torch.Generator().manual_seed(21)
    n = 90 if prompt else 260
    pick = [100, 300, 60, 400, 128, 129, 17, 256] if prompt else [100, 300, 60, 512, 128, 129, 17, 700, 384, 90]
    lens = [pick[int(i)] for i in torch.randint(0, len(pick), (n,), generator=g)]
    new = lens if prompt else [1] * n
    c = Case(lens, new, 8 if prompt else 4, 4, d, 16, seed=22).cuda()
    start = f64(c.weights)
    lse = (torch.randn((c.H, c.total), generator=g) * 0.1 + 6.0).cuda()
    first = weigh(c, lse, out=torch.zeros_like(c.weights))
    check_weights(c, lse, start, first)
    for _ in range(200):
        out = weigh(c, lse, out=torch.zeros_like(c.weights))
        assert torch.equal(out, first)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,H,hkv,slack", [
    ([700], [700], 8, 1, 0),                # 3 tiles: clusters of 4
    ([1100, 300], [1100, 90], 8, 1, 0),     # 10 tiles, 69 chunks: clusters of 8, some CTAs without a chunk
    ([1300, 40], [1300, 30], 16, 2, 0),
    ([2300, 513, 1], [600, 513, 0], 4, 2, 0),    # 60: 4; no new rows in one
    ([700, 300, 130], [700, 300, 130], 14, 2, 40000),  # a large table: clusters of 2
    ([900] * 60, [9] * 60, 128, 1, 0),      # more tiles than the clusters share
])
def test_weights_of_shared_tiles(lens, new, H, hkv, slack, d):
    """Few tiles: clusters share them, and the sums come together in a fixed order."""
    c = Case(lens, new, H, hkv, d, 16, seed=25).cuda()
    c.table = torch.nn.functional.pad(c.table, (0, slack // 16), value=-1).contiguous()
    start = f64(c.weights)
    lse = (torch.randn((H, c.total), generator=torch.Generator().manual_seed(2)) * 0.1 + 6.0).cuda()
    first = weigh(c, lse, out=torch.zeros_like(c.weights))
    check_weights(c, lse, start, first)
    unused = torch.isnan(c.weights)
    assert (first[unused] == 0).all()
    for _ in range(50):
        assert torch.equal(weigh(c, lse, out=torch.zeros_like(c.weights)), first)
    g, outs = torch.cuda.CUDAGraph(), [torch.zeros_like(first) for _ in range(2)]
    with torch.cuda.graph(g):
        for o in outs:
            weigh(c, lse, out=o)
    c.seq_lens.sub_(torch.minimum(c.seq_lens - c.cu.diff(), torch.tensor(3, device="cuda")).clamp(min=0))
    g.replay()
    c.lens = c.seq_lens.tolist()
    check_weights(c, lse, start, outs[0])
    assert torch.equal(outs[0], outs[1])


def test_wait_limit_of_shared_tiles():
    """Copies that never come: every CTA of the cluster gives up and the call returns."""
    c = Case([900], [900], 8, 1, 64, 16, seed=26).cuda()
    lse = torch.full((8, 900), 6.0, device="cuda")
    weigh(c, lse, out=torch.zeros_like(c.weights), options=attn.make_options(timeout_ms=50, test_flags=attn.TEST_WITHHOLD_KV))
    assert attn.get_status() == -8
    first = weigh(c, lse, out=torch.zeros_like(c.weights))
    check_weights(c, lse, f64(c.weights), first)


def test_weights_strided_queries_and_pages():
    H, hkv, d = 6, 2, 64
    c = Case([300, 70], [40, 1], H, hkv, d, 16, seed=4).cuda()
    lse = torch.full((H, c.total), 5.0, device="cuda")
    want = weigh(c, lse, out=torch.zeros_like(c.weights))
    c.q = torch.cat([c.q, c.k_new, c.v_new], 1)[:, :H]
    c.k = c.k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    assert torch.equal(want, weigh(c, lse, out=torch.zeros_like(c.weights)))


# ------------------------------------------------------- append and compact
def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)


@pytest.mark.parametrize("d,hkv,page", [(64, 1, 16), (128, 8, 64), (64, 5, 48), (128, 3, 32)])
@pytest.mark.parametrize("picked", [False, True])
def test_append(d, hkv, page, picked):
    before, new = [0, 7, 100, 63, 5], [5, 0, 1, 70, 2]
    c = Case(before, new, hkv, hkv, d, page, seed=d + hkv, room=80).cuda()
    after = torch.tensor([a + n for a, n in zip(before, new)], dtype=torch.int32, device="cuda")
    pos = after * 3
    rows = torch.randint(0, c.total, (c.total,), dtype=torch.int32).cuda() if picked else None
    want = [x.clone() for x in (c.k, c.v, c.weights, c.positions)]
    for s in range(5):
        for i in range(new[s]):
            at = int(c.cu[s]) + i
            src = int(rows[at]) if picked else at
            slot = before[s] + i
            p, j = int(c.table[s, slot // page]), slot % page
            want[0][p, j], want[1][p, j] = c.k_new[src], c.v_new[src]
            want[2][p, :, j], want[3][p, :, j] = 0.0, int(pos[s]) - new[s] + i
    cache.cache_append(c.k_new, c.v_new, c.k, c.v, c.table, after, c.cu, rows=rows, weights=c.weights,
                       positions=c.positions, seq_pos=pos)
    for w, g in zip(want, (c.k, c.v, c.weights, c.positions)):
        assert torch.equal(bits(w), bits(g))


def test_append_skips_what_does_not_fit():
    c = Case([10, 10], [4, 4], 2, 2, 64, 16, seed=1).cuda()
    k0 = c.k.clone()
    lens = torch.tensor([2, 1 << 30], dtype=torch.int32, device="cuda")   # -2 for the first two; clamped to 16
    rows = torch.tensor([0, 1, 2, 3, 4, -1, 99, 7], dtype=torch.int32, device="cuda")
    c.table[1] = -3
    cache.cache_append(c.k_new, c.v_new, c.k, c.v, c.table, lens, c.cu, rows=rows)
    p = int(c.table[0, 0])
    k0[p, 0], k0[p, 1] = c.k_new[2], c.k_new[3]
    assert torch.equal(bits(k0), bits(c.k))


def do_select(c: Case, budget, recent, pos=None, by_position=True):
    return cache.cache_select(c.weights, c.table, c.seq_lens, budget, recent, c.positions if by_position else None,
                              pos)


@pytest.mark.parametrize("by_position", [True, False])
@pytest.mark.parametrize("lens,hkv,page,budget,recent", [
    ([1, 5, 16], 2, 16, 8, 2), ([100, 300, 64, 65, 0], 3, 48, 64, 16), ([1000, 999, 31], 1, 16, 1, 0),
    ([1025, 4096], 2, 128, 1000, 1000), ([5000], 4, 64, 129, 1), ([700, 129], 2, 32, 128, 128),
])
def test_select(lens, hkv, page, budget, recent, by_position):
    c = Case(lens, [1] * len(lens), hkv, hkv, 64, page, seed=budget)
    g = torch.Generator().manual_seed(budget)
    c.weights = torch.where(torch.rand(c.weights.shape, generator=g) < 0.3, torch.round(c.weights), c.weights)  # ties
    c.positions = torch.randint(0, 2 * max(lens) + 1, c.positions.shape, generator=g, dtype=torch.int32)
    c.cuda()
    pos = c.seq_lens * 2
    kept = do_select(c, budget, recent, pos, by_position)
    assert np.array_equal(kept.cpu().numpy(), ref.select(c, budget, recent, pos.cpu(), by_position))


def test_select_all_equal_and_special_values():
    c = Case([400, 400, 400], [1] * 3, 1, 1, 64, 16, seed=2)
    g = torch.Generator().manual_seed(3)
    vals = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1.0, 3.4e38, 1e-45, -1.0])
    w = vals[torch.randint(0, len(vals), c.weights.shape, generator=g)]
    first = c.table[0][c.table[0] >= 0].long()
    w[first] = 2.5
    c.weights = w
    c.cuda()
    for budget, recent in ((50, 0), (399, 7), (200, 200)):
        kept = do_select(c, budget, recent, by_position=False)
        assert np.array_equal(kept.cpu().numpy(), ref.select(c, budget, recent, by_position=False))


def test_select_longer_than_shared_memory():
    """Weights that do not fit into shared memory are read again in every pass."""
    n, hkv, page = 70001, 2, 128
    c = Case([1], [1], hkv, hkv, 64, page, seed=2)
    blocks = -(-n // page)
    g = torch.Generator().manual_seed(4)
    c.n_pages = blocks
    c.table = torch.randperm(blocks, generator=g).to(torch.int32).view(1, -1)
    c.weights = torch.round(torch.rand((blocks, hkv, page), generator=g) * 1000)
    c.positions = torch.randint(0, n, (blocks, hkv, page), generator=g, dtype=torch.int32)
    c.lens, c.seq_lens = [n], torch.tensor([n], dtype=torch.int32)
    for name in ("table", "weights", "positions", "seq_lens"):
        setattr(c, name, getattr(c, name).cuda())
    pos = torch.tensor([n], dtype=torch.int32, device="cuda")
    for budget in (1, 9999, 60000, 70000):
        recent = min(budget, 500)
        kept = do_select(c, budget, recent, pos)
        assert np.array_equal(kept.cpu().numpy(), ref.select(c, budget, recent, pos.cpu()))


@pytest.mark.parametrize("d,hkv,page", [(64, 2, 16), (128, 3, 48), (64, 1, 64), (128, 8, 128)])
@pytest.mark.parametrize("budget", [5, 64, 257])
def test_evict(d, hkv, page, budget):
    lens = [300, 64, 1, 900, 258]
    c = Case(lens, [1] * 5, hkv, hkv, d, page, seed=budget).cuda()
    pos = c.seq_lens.clone()
    recent = budget // 4
    want_kept = ref.select(c, budget, recent, pos.cpu())
    want = [x.clone() for x in (c.k, c.v, c.weights, c.positions)]
    tab = c.table.cpu()
    for s in range(5):
        for h in range(hkv):
            for i in range(min(budget, lens[s])):
                f = int(want_kept[s, h, i])
                if f != i:
                    a, b = (int(tab[s, f // page]), f % page), (int(tab[s, i // page]), i % page)
                    want[0][b[0], b[1], h], want[1][b[0], b[1], h] = c.k[a[0], a[1], h], c.v[a[0], a[1], h]
                    want[2][b[0], h, b[1]], want[3][b[0], h, b[1]] = c.weights[a[0], h, a[1]], c.positions[a[0], h, a[1]]
    kept = cache.cache_evict(c.k, c.v, c.weights, c.table, c.seq_lens, budget, recent, c.positions, pos)
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    for w, g in zip(want, (c.k, c.v, c.weights, c.positions)):
        assert torch.equal(bits(w), bits(g))


def test_compact_skips_entries_outside():
    c = Case([40], [1], 1, 1, 64, 16, seed=3).cuda()
    k0, v0 = c.k.clone(), c.v.clone()
    kept = torch.tensor([[[-1, 3, 1 << 30, 48, 2, 39]]], dtype=torch.int32, device="cuda")  # budget 6; 48 = capacity
    cache.cache_compact(kept, c.k, c.v, c.table)
    p, q = int(c.table[0, 0]), int(c.table[0, 2])
    k0[p, 5], v0[p, 5] = k0[q, 7], v0[q, 7]
    assert torch.equal(bits(k0), bits(c.k)) and torch.equal(bits(v0), bits(c.v))


# -------------------------------------------------- streams, graphs, together
def test_on_another_stream():
    c = Case([3000, 70], [4, 2], 8, 2, 128, 32, seed=20).cuda()
    lse0 = torch.full((8, c.total), 6.0, device="cuda")
    want = attend(c)
    want_w = weigh(c, lse0, out=torch.zeros_like(c.weights))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        got = attend(c, stream=s)
        w = torch.zeros_like(c.weights)
        s.wait_stream(torch.cuda.current_stream())
        weigh(c, lse0, out=w, stream=s)
        junk = [torch.full((1 << 20,), 9.0, device="cuda") for _ in range(4)]  # reuses what the calls freed
        s.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and torch.equal(want_w, w)
        del junk


def test_two_streams_at_once():
    """Attention and weights side by side (both want the SMs' tensor memory)."""
    a = Case([5000, 300], [60, 2], 8, 2, 128, 64, seed=23).cuda()
    b = Case([4000, 900], [4000, 1], 8, 2, 64, 16, seed=24).cuda()
    lse = torch.full((8, b.total), 7.0, device="cuda")
    want, want_w = attend(a), weigh(b, lse, out=torch.zeros_like(b.weights))
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        w = torch.zeros_like(b.weights)
        t.wait_stream(torch.cuda.current_stream())
        got = attend(a, stream=s)
        weigh(b, lse, out=w, stream=t)
        again = attend(a, stream=t)
        torch.cuda.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and torch.equal(want_w, w)
        assert torch.equal(want[0], again[0])


def test_two_graphs_share_a_workspace():
    """Two captured steps over one workspace, replayed in turn with other lengths,
    tables and trees than at the capture."""
    a = Case([900, 30], [3, 1], 8, 2, 64, 16, seed=21, room=8).cuda()
    b = Case([10, 500], [2, 60], 8, 2, 64, 16, seed=22).cuda()
    ws = torch.empty(cache.workspace_size(8, 2, 64, 64), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for c in (a, b):
        attend(c, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(attend(c, workspace=ws))
        graphs.append(g)
    for turn in range(3):
        for c, g, o in ((a, graphs[0], outs[0]), (b, graphs[1], outs[1])):
            o[0].fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            check_attention(c, *o)
        # shorter sequences, another tree and other rows for the next turn
        for c in (a, b):
            c.lens = [max(0, n - 5 * (turn + 1)) for n in c.lens]
            c.seq_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
            c.q.copy_(torch.randn(c.q.shape).bfloat16())
            c.parents.fill_(-1)


def test_step_in_a_graph():
    """Attention, append, weights, selection and compaction captured once and
    replayed with other lengths, trees and rows: as the same calls made directly."""
    H, hkv, d, page, budget = 4, 2, 64, 16, 40
    base = Case([100, 33, 70], [4, 4, 4], H, hkv, d, page, seed=31, room=8).cuda()
    base.positions.clamp_(min=0)
    rows = torch.tensor([0, 1, 4, 8, 9, 11], dtype=torch.int32, device="cuda")
    cu_acc = torch.tensor([0, 2, 3, 6], dtype=torch.int32, device="cuda")
    names = ("k", "v", "weights", "positions", "seq_lens", "q", "k_new", "v_new", "parents", "table")

    def step(s):
        o, lse = cache.attn_fwd_cache(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["seq_lens"],
                                      base.cu, 4, parents=s["parents"])
        after = s["seq_lens"] + (cu_acc[1:] - cu_acc[:-1])
        cache.cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], after, cu_acc, rows=rows,
                           weights=s["weights"], positions=s["positions"], seq_pos=after)
        r = rows.long()
        cache.cache_weights(s["q"][r], lse[:, r].contiguous(), s["k"], s["table"], after, cu_acc, 3, s["weights"])
        kept = cache.cache_evict(s["k"], s["v"], s["weights"], s["table"], after, budget, 8, s["positions"], after)
        return o, lse, kept

    live = {n: getattr(base, n).clone() for n in names}
    step({n: t.clone() for n, t in live.items()})
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(live)
    for turn, lens in enumerate(([100, 33, 70], [41, 0, 39], [7, 33, 64])):
        state = {n: getattr(base, n).clone() for n in names}
        state["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        state["parents"].fill_(-1 if turn else 0)
        state["q"].copy_(torch.randn(state["q"].shape).bfloat16())
        for n in names:
            live[n].copy_(state[n])
        want = step(state)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
        for n in ("k", "v", "weights", "positions"):
            assert torch.equal(bits(state[n]), bits(live[n])), (turn, n)


def test_offsets_beyond_32_bits():
    """Pages more than 2^32 elements from the first."""
    hkv, d, page, n_pages = 8, 128, 64, 70000
    assert n_pages * page * hkv * d > 1 << 32
    k = torch.empty((n_pages, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    w = torch.zeros((n_pages, hkv, page), device="cuda")
    pos = torch.zeros((n_pages, hkv, page), dtype=torch.int32, device="cuda")
    c = Case([0], [1], 8, hkv, d, page, seed=32).cuda()
    n = 100
    g = torch.Generator().manual_seed(33)
    table = torch.tensor([[n_pages - 1, n_pages - 7]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    kn, vn = (torch.randn((n, hkv, d), generator=g).bfloat16().cuda() for _ in range(2))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    cache.cache_append(kn, vn, k, v, table, lens, cu, weights=w, positions=pos)
    assert torch.equal(k[n_pages - 1], kn[:64]) and torch.equal(v[n_pages - 7, :36], vn[64:])
    # the same keys in a small cache
    c.lens, c.seq_lens, c.n_pages = [n], lens, 2
    c.table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    c.k, c.v = (torch.stack([t[n_pages - 7], t[n_pages - 1]]) for t in (k, v))
    o, lse = cache.attn_fwd_cache(c.q, c.k_new, c.v_new, k, v, table, lens, c.cu, 1)
    c.parents = None
    check_attention(c, o, lse)
    cache.cache_weights(c.q, lse, k, table, lens, c.cu, 1, w)
    c.weights = torch.stack([w[n_pages - 7], w[n_pages - 1]])
    check_weights(c, lse, np.zeros(c.weights.shape), c.weights)
    kept = cache.cache_evict(k, v, w, table, lens, 50, 0)
    moved = kept[0, 3].tolist()
    for i in range(50):
        assert torch.equal(k[n_pages - 1, i, 3], kn[moved[i], 3]) and torch.equal(v[n_pages - 1, i, 3], vn[moved[i], 3])


def test_generation_with_drafts_and_eviction():
    """A prompt, then steps of drafting, attention, acceptance, append, weights and
    eviction, as they are used together, against the definitions on plain lists."""
    H, hkv, d, page, budget, recent = 4, 2, 64, 16, 96, 24
    G, scale = H // hkv, d ** -0.5
    g = torch.Generator().manual_seed(30)
    lens = [200, 45]
    n_seq, blocks = 2, 20
    table = torch.randperm(n_seq * blocks, generator=g).to(torch.int32).view(n_seq, blocks).cuda()
    n_pages = n_seq * blocks
    kc = torch.full((n_pages, page, hkv, d), float("nan"), device="cuda").bfloat16()
    vc = kc.clone()
    wts = torch.full((n_pages, hkv, page), float("nan"), device="cuda")
    pos = torch.zeros((n_pages, hkv, page), dtype=torch.int32, device="cuda")
    rnd = lambda *sh: torch.randn(sh, generator=g).bfloat16()  # noqa: E731
    # plain state: per sequence and head lists of (k, v, weight, position)
    plain = [[[] for _ in range(hkv)] for _ in range(n_seq)]

    def check_state(seq_lens):
        kk, vv, ww, pp, tt = f64(kc), f64(vc), f64(wts), pos.cpu().numpy(), table.cpu()
        for s in range(n_seq):
            for h in range(hkv):
                L = plain[s][h]
                assert len(L) == int(seq_lens[s])
                for j, (k, v, w, p) in enumerate(L):
                    pg, i = int(tt[s, j // page]), j % page
                    assert np.array_equal(kk[pg, i, h], k) and np.array_equal(vv[pg, i, h], v)
                    assert pp[pg, h, i] == p and abs(ww[pg, h, i] - w) <= 1e-5 * (1 + abs(w))

    def add_weights(s, qs, lses):
        n = len(qs)
        for h in range(hkv):
            L = plain[s][h]
            K = np.array([e[0] for e in L])
            w = np.zeros(len(L))
            for i in range(n):
                for gq in range(G):
                    p = np.exp(K @ qs[i, h * G + gq] * scale - lses[h * G + gq, i])
                    p[len(L) - n + i + 1:] = 0
                    w += p
            plain[s][h] = [(k, v, a + x, p) for (k, v, a, p), x in zip(L, w)]

    # the prompt: the library's packed attention, then append and weights
    cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    q, k, v = (rnd(sum(lens), n, d).cuda() for n in (H, hkv, hkv))
    _, lse = attn.attn_fwd_varlen(q, k, v, cu, cu, max(lens), causal=True)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    seq_pos = seq_lens.clone()
    cache.cache_append(k, v, kc, vc, table, seq_lens, cu, weights=wts, positions=pos, seq_pos=seq_pos)
    cache.cache_weights(q, lse, kc, table, seq_lens, cu, max(lens), wts)
    for s in range(n_seq):
        r = slice(int(cu[s]), int(cu[s + 1]))
        for h in range(hkv):
            plain[s][h] = [(f64(k)[j, h], f64(v)[j, h], 0.0, j - r.start) for j in range(r.start, r.stop)]
        add_weights(s, f64(q)[r], f64(lse)[:, r])
    check_state(seq_lens)

    for step in range(4):
        # eviction
        before = seq_lens.cpu().numpy()
        cache.cache_evict(kc, vc, wts, table, seq_lens, budget, recent, pos, seq_pos)
        seq_lens.clamp_(max=budget)
        ww, tt = f64(wts), table.cpu()
        for s in range(n_seq):
            for h in range(hkv):
                L = plain[s][h]
                w = np.array([e[2] for e in L])
                new = np.array([e[3] >= int(seq_pos[s]) - recent for e in L])
                kp = ref.selected(w, new, budget)
                plain[s][h] = [L[j] for j in kp if j >= 0]
        check_state(seq_lens)
        # drafts
        new = [7, 4]
        cu = torch.tensor([0, 7, 11], dtype=torch.int32, device="cuda")
        parents = torch.tensor([-1, 0, 0, 1, 1, 3, -1] + [-1, 0, 1, 1], dtype=torch.int32, device="cuda")
        q, k, v = (rnd(11, n, d).cuda() for n in (H, hkv, hkv))
        o, lse = cache.attn_fwd_cache(q, k, v, kc, vc, table, seq_lens, cu, 7, parents=parents)
        for s, r in enumerate((slice(0, 7), slice(7, 11))):
            seen = ref.ancestors(parents[r].cpu().numpy(), new[s])
            for hq in range(H):
                L = plain[s][hq // G]
                K = np.concatenate([np.array([e[0] for e in L]), f64(k)[r, hq // G]])
                V = np.concatenate([np.array([e[1] for e in L]), f64(v)[r, hq // G]])
                z = f64(q)[r, hq] @ K.T * scale
                z[:, len(L):][~seen] = -np.inf
                l = np.log(np.exp(z).sum(1))
                p = np.exp(z - l[:, None])
                tol = HALF_BF16 * 2.02 * (p @ np.abs(V)) + 1e-4
                assert (np.abs(f64(o)[r, hq] - p @ V) <= tol).all()
                assert (np.abs(f64(lse)[hq, r] - l) <= 1e-4).all()
        # the accepted paths: 0 -> 1 -> 3 -> 5 and 0 -> 1
        paths = ([0, 1, 3, 5], [7, 8])
        rows = torch.tensor(paths[0] + paths[1], dtype=torch.int32, device="cuda")
        cu_acc = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
        n_acc = torch.tensor([4, 2], dtype=torch.int32, device="cuda")
        seq_lens += n_acc
        seq_pos += n_acc
        cache.cache_append(k, v, kc, vc, table, seq_lens, cu_acc, rows=rows, weights=wts, positions=pos,
                           seq_pos=seq_pos)
        qa, la = q[rows.long()], lse[:, rows.long()].contiguous()
        cache.cache_weights(qa, la, kc, table, seq_lens, cu_acc, 4, wts)
        for s, r in enumerate((slice(0, 4), slice(4, 6))):
            for h in range(hkv):
                at = int(seq_pos[s]) - len(paths[s])
                plain[s][h] += [(f64(k)[j, h], f64(v)[j, h], 0.0, at + i) for i, j in enumerate(paths[s])]
            add_weights(s, f64(qa)[r], f64(la)[:, r])
        check_state(seq_lens)


def test_both_ways_to_the_library_agree():
    """A named stream takes the general way, dense tensors without one the short way."""
    import sys

    c = Case([90, 33, 0], [3, 1, 2], 4, 2, 64, 16, seed=41, room=3).cuda()
    here = torch.cuda.current_stream()
    lens = c.seq_lens + (c.cu[1:] - c.cu[:-1])
    rows = torch.arange(c.total - 1, -1, -1, dtype=torch.int32, device="cuda")

    def state():
        return [t.clone() for t in (c.k, c.v, torch.nan_to_num(c.weights), c.positions)]

    for scale in (None, 0.25):
        for parents in (None, c.parents):
            ways = [cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 3, parents=parents,
                                         scale=scale, stream=s) for s in (None, here)]
            o, lse = ways[0]
            assert torch.equal(o, ways[1][0]) and torch.equal(lse, ways[1][1])
        out, ls = torch.empty_like(o), torch.empty_like(lse)
        ws = torch.empty(cache.workspace_size(4, 2, 3, 64), dtype=torch.uint8, device="cuda")
        refs = [sys.getrefcount(t) for t in (out, ls, ws, c.q, c.table)]
        got = cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 3, parents=c.parents,
                                   scale=scale, out=out, lse=ls, workspace=ws)
        assert got[0] is out and got[1] is ls and torch.equal(out, o) and torch.equal(ls, lse)
        del got
        assert refs == [sys.getrefcount(t) for t in (out, ls, ws, c.q, c.table)]
        w0 = torch.rand_like(c.weights)
        a = cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 3, w0, scale=scale, out=w0.clone())
        b = cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 3, w0, scale=scale, out=w0.clone(), stream=here)
        assert torch.equal(a, b)

    w = torch.rand_like(c.weights)
    for kw in (dict(positions=c.positions, seq_pos=c.seq_lens), dict()):
        kept = [cache.cache_select(w, c.table, c.seq_lens, 20, 4, stream=s, **kw) for s in (None, here)]
        assert torch.equal(*kept)
        given = torch.empty_like(kept[0])
        assert cache.cache_select(w, c.table, c.seq_lens, 20, 4, kept=given, **kw) is given
        assert torch.equal(given, kept[0])

    first = [t.clone() for t in (c.k, c.v, c.weights, c.positions)]
    results = []
    for s in (None, here):
        for t, t0 in zip((c.k, c.v, c.weights, c.positions), first):
            t.copy_(t0)
        cache.cache_append(c.k_new, c.v_new, c.k, c.v, c.table, lens, c.cu, rows=rows, weights=c.weights,
                           positions=c.positions, seq_pos=lens, stream=s)
        cache.cache_compact(kept[0], c.k, c.v, c.table, c.weights, c.positions, stream=s)
        results.append(state())
    for x, y in zip(*results):
        assert torch.equal(bits(x), bits(y))
    for f, args in ((cache.cache_select, (w, c.table, c.seq_lens, 8, 9)),
                    (cache.cache_append, (c.k_new, c.v_new, c.k.view(-1, 8, 2, 64), c.v.view(-1, 8, 2, 64), c.table,
                                          c.seq_lens, c.cu))):
        for s in (None, here):
            with pytest.raises(attn.AttnError):
                f(*args, stream=s)


def test_binding_refuses_what_does_not_fit():
    """Wrong types, shapes, devices and strides are ValueErrors that name the tensor."""
    c = Case([40, 20], [2, 1], 4, 2, 64, 16, seed=40).cuda()
    lse = torch.zeros((4, 3), device="cuda")
    kept = torch.zeros((2, 2, 8), dtype=torch.int32, device="cuda")
    attend_args = dict(q=c.q, k_new=c.k_new, v_new=c.v_new, k_cache=c.k, v_cache=c.v, block_table=c.table,
                       seq_lens=c.seq_lens, cu_seqlens_q=c.cu, max_seqlen_q=2, parents=c.parents)
    calls = {
        cache.attn_fwd_cache: attend_args,
        cache.cache_append: dict(k_new=c.k_new, v_new=c.v_new, k_cache=c.k, v_cache=c.v, block_table=c.table,
                                 seq_lens=c.seq_lens, cu_new=c.cu, weights=c.weights, positions=c.positions,
                                 seq_pos=c.seq_lens),
        cache.cache_weights: dict(q=c.q, lse=lse, k_cache=c.k, block_table=c.table, seq_lens=c.seq_lens,
                                  cu_seqlens_q=c.cu, max_seqlen_q=2, weights=c.weights),
        cache.cache_select: dict(weights=c.weights, block_table=c.table, seq_lens=c.seq_lens, budget=8,
                                 positions=c.positions, seq_pos=c.seq_lens),
        cache.cache_compact: dict(kept=kept, k_cache=c.k, v_cache=c.v, block_table=c.table, weights=c.weights,
                                  positions=c.positions),
    }
    before = [t.clone() for t in (c.k, c.v, c.weights, c.positions)]
    for f, args in calls.items():
        for name, t in args.items():
            if not isinstance(t, torch.Tensor):
                continue
            bad = [t.cpu(), t.to(torch.float16 if t.dtype.is_floating_point else torch.int64), t[..., None], 3,
                   t.repeat(*([1] * (t.dim() - 1) + [2]))[..., ::2]]
            if t.dim() == 1:
                bad.append(torch.cat([t, t]))
            if name not in ("parents", "weights", "positions", "seq_pos"):
                bad.append(None)
            for x in bad:
                with pytest.raises(ValueError):
                    f(**{**args, name: x})
    with pytest.raises(ValueError):  # 5 heads over 2
        cache.attn_fwd_cache(**{**attend_args, "q": torch.zeros((3, 5, 64), device="cuda").bfloat16()})
    with pytest.raises(attn.AttnError) as e:
        cache.attn_fwd_cache(**{**attend_args, "max_seqlen_q": 129})
    assert e.value.code == -2
    with pytest.raises(attn.AttnError) as e:
        cache.cache_select(c.weights, c.table, c.seq_lens, 0)
    assert e.value.code == -2
    torch.cuda.synchronize()
    for a, b in zip(before, (c.k, c.v, c.weights, c.positions)):
        assert torch.equal(bits(a), bits(b))
