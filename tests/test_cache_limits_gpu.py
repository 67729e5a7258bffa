"""Calls at the edges of what the cache operators' contract allows, on the GPU."""

from __future__ import annotations

import os
import random
import subprocess
import sys
import textwrap
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import cache_reference as ref
from cache_reference import HALF_F32, Case, f64
from exact_attention_63_gb300 import attn, build, cache
from gpu_common import need_gpu
from test_cache_gpu import bits, check_attention, check_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    need_gpu()
    assert attn.get_status() == 0
    yield
    assert attn.get_status() == 0


@pytest.mark.parametrize("most", [8, 33, 40, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_fewer_tokens_than_max_seqlen(d, most):
    """max_seqlen is a bound: above total, and above every sequence's tokens."""
    c = Case([300, 40, 129], [3, 1, 4], 8, 2, d, 16, seed=50).cuda()
    args = (c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu)
    ws = torch.empty(cache.workspace_size(8, 2, 128, d), dtype=torch.uint8, device="cuda")  # for every max_seqlen
    for kw in (dict(), dict(workspace=ws), dict(stream=torch.cuda.current_stream())):
        o, lse = cache.attn_fwd_cache(*args, most, parents=c.parents, **kw)
        check_attention(c, o, lse)


def test_attention_of_one_full_row_tile_with_room_for_two():
    """30 rows of 4 heads under a bound of 40: total decides on one row tile a CTA, which leaves more
    parts than two would."""
    c = Case([700], [30], 8, 2, 128, 16, seed=51).cuda()
    for kw in (dict(), dict(stream=torch.cuda.current_stream())):
        o, lse = cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 40, parents=c.parents, **kw)
        check_attention(c, o, lse)


def test_wait_limit_where_a_loader_is_done():
    """One chunk of rows a tile: the rows' loader has issued all its copies when the waits for the
    withheld keys run out.  Each call ends, and the next one is right."""
    c = Case([200, 90, 256], [1, 2, 1], 8, 2, 128, 16, seed=52).cuda()
    start, lse = f64(c.weights), torch.full((8, c.total), 6.0, device="cuda")
    opts = attn.make_options(timeout_ms=1, test_flags=attn.TEST_WITHHOLD_KV)
    for i in range(10):
        lse[:, 1] = float("inf") if i % 2 else 6.0
        cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 2, c.weights, out=torch.zeros_like(c.weights), options=opts)
        assert attn.get_status() == -8
        out = cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 2, c.weights, out=torch.zeros_like(c.weights))
        check_weights(c, lse, start, out)


def test_weights_where_no_cluster_fits(tmp_path):
    """Sharing a tile is a matter of speed: where the runtime knows of no cluster that fits (here a stand-in for
    its query that fails and leaves an error behind), single CTAs do the work, and the calls after it are right."""
    home = build.cuda_home(build.nvcc_path())
    source, fake = tmp_path / "fake.cpp", tmp_path / "fake.so"
    source.write_text(textwrap.dedent("""
        extern "C" int cudaSetDevice(int);
        extern "C" int cudaOccupancyMaxActiveClusters(int* n, const void*, const void*) {
          *n = 0;
          return cudaSetDevice(99999);
        }
    """))
    subprocess.run(["g++", "-shared", "-fPIC", str(source), "-o", str(fake), f"-L{home}/lib64", "-lcudart"], check=True)
    program = textwrap.dedent("""
        import torch
        from cache_reference import Case, f64
        from exact_attention_63_gb300 import attn, cache
        from test_cache_gpu import check_attention, check_weights, attend
        c = Case([900], [900], 8, 1, 64, 16, seed=53).cuda()
        lse = torch.full((8, 900), 6.0, device="cuda")
        for _ in range(2):
            out = cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 900, c.weights, out=torch.zeros_like(c.weights))
            cache.cache_append(c.k_new, c.v_new, c.k.clone(), c.v.clone(), c.table, c.seq_lens, c.cu)
            check_weights(c, lse, f64(c.weights), out)
        assert attn.get_status() == 0
        print("fine")
    """)
    tests = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, LD_PRELOAD=str(fake), PYTHONPATH=os.pathsep.join((os.path.dirname(tests), tests)))
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def weigh(c: Case, lse, **kw):
    return cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, c.max_new(), c.weights, **kw)


@pytest.mark.parametrize("d", [64, 128])
def test_weights_at_the_smallest_scale(d):
    """scale = 1e-30 with queries and keys of 1e15: scores of ordinary size, -LSE/scale of 1e31."""
    c = Case([300, 70], [40, 70], 4, 2, d, 16, seed=54)
    c.weights = torch.nan_to_num(c.weights)
    size = (c.d + 8) * HALF_F32 * max(float(c.q.float().norm(dim=-1).max()) * float(c.k.float().nan_to_num().norm(dim=-1).max()), 8)
    c.q, c.k, c.scale = (c.q.float() * 1e15).bfloat16(), (c.k.float() * 1e15).bfloat16(), 1.0000001e-30
    c.cuda()
    lse = (torch.randn((4, c.total), generator=torch.Generator().manual_seed(3)) + 7).cuda()
    W, start = ref.weights(c, lse, f64(c.weights)), f64(c.weights)
    got, used = f64(weigh(c, lse, scale=c.scale, out=torch.zeros_like(c.weights))), ~np.isnan(W)
    # scores off by `size` (fp32 sums of |q||k|) and the rounding of scale, -LSE/scale in three terms of bf16; fp32 sums
    tol = (4 * size + 2.0 ** -15) * (W - start) + 2.0 ** -22 * W + 1e-30
    assert (np.abs(got - W) <= tol)[used].all()


def test_weights_of_extreme_lse():
    """Finite LSEs far from any score, up to the largest: nothing is added, or infinity."""
    c = Case([200, 130], [3, 130], 4, 2, 64, 16, seed=55).cuda()
    start = f64(c.weights)
    lse = torch.full((4, c.total), 5.0, device="cuda")
    top = torch.finfo(torch.float32).max
    for value in (1e9, 4.2e37, 4.25e37, 3.4e38, top):  # (over the scale of 1/8: within bf16, within fp32 only, beyond)
        lse[0, 1::3] = value
        check_weights(c, lse, start, weigh(c, lse, out=torch.zeros_like(c.weights)))
        low = lse.clone()
        low[0, 4] = -value
        W = ref.weights(c, low, start)
        got = f64(weigh(c, low, out=torch.zeros_like(c.weights)))
        assert np.array_equal(np.isinf(W), np.isinf(got) & ~np.isnan(W)) and not np.isnan(got).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,H,hkv", [([1100, 300], [1100, 90], 8, 1), ([900] * 20, [33] * 20, 12, 3), ([5000, 77], [1, 2], 8, 2)])
def test_weights_of_rows_left_out(lens, new, H, hkv, d):
    """An infinite LSE leaves its row out, whatever the row's query holds (the padding of a batch of fixed
    shape): whole chunks of such rows, some in a chunk, with keys that have no weight in them."""
    c = Case(lens, new, H, hkv, d, 16, seed=56).cuda()
    g = torch.Generator().manual_seed(57)
    start = f64(c.weights)
    lse = (torch.randn((H, c.total), generator=g) * 0.1 + 6.0).cuda()
    off = (torch.rand(c.total, generator=g) < 0.2).cuda()
    off[: min(70, c.total // 2)] = True
    lse[:, off] = float("inf")
    lse[0, ::7] = -float("inf")  # (one head of some: its query alone is left out)
    clean = weigh(c, lse, out=torch.zeros_like(c.weights))
    check_weights(c, lse, start, clean)
    for junk in (float("nan"), float("inf"), torch.finfo(torch.bfloat16).max):
        c.q[off] = junk
        c.q[::7, 0] = junk
        assert torch.equal(weigh(c, lse, out=torch.zeros_like(c.weights)), clean)


def test_a_step_without_tokens():
    """No sequence has a new token: every operator takes it, and the weights are what they were."""
    c = Case([40, 0, 300], [0, 0, 0], 4, 2, 64, 16, seed=58).cuda()
    here = torch.cuda.current_stream()
    before = [t.clone() for t in (c.k, c.v, c.weights, c.positions)]
    used = ~torch.isnan(c.weights)
    for stream in (None, here):
        o, lse = cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 1, stream=stream)
        assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
        cache.cache_append(c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, weights=c.weights, positions=c.positions,
                           stream=stream)
        for most in (0, 1, 5):
            args = (c.q, lse, c.k, c.table, c.seq_lens, c.cu, most)
            assert cache.cache_weights(*args, c.weights, stream=stream) is c.weights
            out = torch.full_like(c.weights, 5.0)
            assert cache.cache_weights(*args, c.weights, out=out, stream=stream) is out
            assert torch.equal(out[used], c.weights[used]) and (out[~used] == 5).all()
            assert cache.cache_weights(*args, out=out, stream=stream) is out
            assert (out[used] == 0).all() and (out[~used] == 5).all()
    for a, b in zip(before, (c.k, c.v, c.weights, c.positions)):
        assert torch.equal(bits(a), bits(b))
    with pytest.raises(ValueError):
        cache.cache_weights(c.q, lse[:3], c.k, c.table, c.seq_lens, c.cu, 0, c.weights)


def test_an_empty_step_in_a_graph():
    c = Case([40, 300], [0, 0], 4, 2, 64, 16, seed=59).cuda()
    lse, out = torch.zeros((4, 0), device="cuda"), torch.zeros_like(c.weights)
    cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 0, c.weights, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 0, c.weights, out=out)
    c.weights += 1
    for _ in range(2):
        out.zero_()
        g.replay()
        used = ~torch.isnan(c.weights)
        assert torch.equal(out[used], c.weights[used])


def test_outputs_and_workspaces_that_do_not_fit():
    c = Case([40, 20], [2, 1], 4, 2, 64, 16, seed=60).cuda()
    args = (c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 2)
    o, lse = cache.attn_fwd_cache(*args)
    ws = torch.zeros(cache.workspace_size(4, 2, 2, 64) + 512, dtype=torch.uint8, device="cuda")
    for bad in (3, "ws", ws.cpu(), ws[::2]):
        with pytest.raises(ValueError):
            cache.attn_fwd_cache(*args, workspace=bad)
    for bad in (ws[16:], ws[256:-513]):
        with pytest.raises(attn.AttnError) as e:
            cache.attn_fwd_cache(*args, workspace=bad)
        assert e.value.code == -10
    for name, t in (("out", o), ("lse", lse)):
        for bad in (3, t.cpu(), t.double(), t[:-1], t[None], t.transpose(0, 1)):
            with pytest.raises(ValueError):
                cache.attn_fwd_cache(*args, **{name: bad})
    with pytest.raises(ValueError):
        cache.cache_select(torch.nan_to_num(c.weights), c.table, c.seq_lens, 8, kept=[1])
    assert torch.equal(cache.attn_fwd_cache(*args, workspace=ws[256:-256])[0], o)


# ------------------------------------------------ values out of range, with margins around every output
class Guarded:
    """A tensor inside a larger buffer whose margins hold `fill`."""

    MARGIN = 4096

    def __init__(self, shape, dtype, fill):
        n = int(np.prod(shape))
        self.fill = fill
        self.buffer = torch.full((n + 2 * self.MARGIN,), fill, dtype=dtype, device="cuda")
        self.t = self.buffer[self.MARGIN:self.MARGIN + n].view(shape)

    def intact(self):
        return bool((self.buffer[:self.MARGIN] == self.fill).all() and (self.buffer[-self.MARGIN:] == self.fill).all())


def malformed(H, hkv, d, page, seed):
    """(the case as given, the same with every value clamped into its range): lengths, pages and offsets beyond
    both ends, more rows of a sequence than max_seqlen, rows behind the last one.  All slots hold numbers."""
    c = Case([5 * page, 3 * page, 2 * page + 1, 9], [2, 3, 1, 1], H, hkv, d, page, seed=seed, slack=4)
    g = torch.Generator().manual_seed(seed)
    c.k, c.v = (torch.randn(t.shape, generator=g).bfloat16() for t in (c.k, c.v))
    c.weights = torch.rand(c.weights.shape, generator=g)
    c.positions = torch.randint(0, 99, c.positions.shape, generator=g, dtype=torch.int32)
    c.cuda()
    n, cap = c.n_pages, c.table.shape[1] * page
    # pages 0 and n - 1 stand for the bad ones: no sequence has them, and none of the others is in use twice
    c.table[:] = torch.arange(1, c.table.numel() + 1, device="cuda").view(c.table.shape) % (n - 2) + 1
    c.table[0, 1], c.table[0, 3], c.table[1, 0], c.table[2, 2] = -5, 1 << 30, n, -(1 << 31)
    c.seq_lens[:] = torch.tensor([(1 << 31) - 1, -4, 2 * page + 1, 9], dtype=torch.int32, device="cuda")
    c.cu[:] = torch.tensor([-3, 2, 5, 6, 900], dtype=torch.int32, device="cuda")
    good = {"table": c.table.clamp(0, n - 1), "seq_lens": c.seq_lens.clamp(0, cap), "cu": c.cu.clamp(0, c.total)}
    return c, good


@pytest.mark.parametrize("H,hkv,d,page", [(8, 2, 64, 16), (6, 2, 128, 48), (64, 1, 128, 32)])
def test_attention_of_malformed_values_is_that_of_clamped_ones(H, hkv, d, page):
    c, good = malformed(H, hkv, d, page, seed=61)
    results = []
    for v in ({}, good):
        o, lse = Guarded((c.total, H, d), torch.bfloat16, 7.0), Guarded((H, c.total), torch.float32, 7.0)
        ws = Guarded((cache.workspace_size(H, hkv, 2, d),), torch.uint8, 171)
        k0, v0 = c.k.clone(), c.v.clone()
        cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, v.get("table", c.table), v.get("seq_lens", c.seq_lens),
                             v.get("cu", c.cu), 2, parents=c.parents, out=o.t, lse=lse.t, workspace=ws.t)
        assert o.intact() and lse.intact() and ws.intact()
        assert torch.equal(bits(k0), bits(c.k)) and torch.equal(bits(v0), bits(c.v))
        assert (o.t[4] == 7).all() and (lse.t[:, 4] == 7).all()  # the second sequence's third row: beyond max_seqlen
        results.append((o.t, lse.t))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    assert torch.isfinite(results[0][0]).all()


@pytest.mark.parametrize("H,hkv,d,page", [(8, 2, 64, 16), (6, 2, 128, 48), (64, 1, 128, 32)])
def test_weights_of_malformed_values(H, hkv, d, page):
    """As with clamped lengths and offsets; what lies on a page that is not there is left alone."""
    c, good = malformed(H, hkv, d, page, seed=62)
    lse = torch.full((H, c.total), 5.0, device="cuda")
    outs = []
    for v in ({}, good):
        out = Guarded(c.weights.shape, torch.float32, -3.0)
        cache.cache_weights(c.q, lse, c.k, v.get("table", c.table), v.get("seq_lens", c.seq_lens), v.get("cu", c.cu), 2,
                            c.weights, out=out.t)
        assert out.intact()
        outs.append(out.t)
    assert (outs[0][0] == -3).all() and (outs[0][-1] == -3).all()
    assert torch.equal(outs[0][1:-1], outs[1][1:-1])
    assert (outs[0] != -3).any()


@pytest.mark.parametrize("budget", [3, 40, 1000])
def test_selection_and_compaction_of_malformed_values(budget):
    c, good = malformed(8, 2, 64, 16, seed=63)
    kept = []
    for v in ({}, good):
        out = Guarded((4, 2, budget), torch.int32, 77)
        cache.cache_select(c.weights, v.get("table", c.table), v.get("seq_lens", c.seq_lens), budget, 2, c.positions,
                           c.seq_lens.clamp(0, 99), kept=out.t)
        assert out.intact()
        kept.append(out.t)
    assert torch.equal(*kept)
    # moves from or to a page that is not there are skipped, and nothing else than the moves changes
    state = [Guarded(t.shape, t.dtype, 5) for t in (c.k, c.v, c.weights, c.positions)]
    for s, t in zip(state, (c.k, c.v, c.weights, c.positions)):
        s.t.copy_(t)
    cache.cache_compact(kept[0], state[0].t, state[1].t, c.table, state[2].t, state[3].t)
    assert all(s.intact() for s in state)
    want, tab = [t.clone() for t in (c.k, c.v, c.weights, c.positions)], c.table.tolist()
    there = lambda s, j: j // 16 < len(tab[s]) and 0 <= tab[s][j // 16] < c.n_pages  # noqa: E731
    for s in range(4):
        for h in range(2):
            for i, j in enumerate(kept[0][s, h].tolist()):
                if j >= budget and there(s, i) and there(s, j):
                    a, b = (tab[s][j // 16], j % 16), (tab[s][i // 16], i % 16)
                    want[0][b[0], b[1], h], want[1][b[0], b[1], h] = c.k[a[0], a[1], h], c.v[a[0], a[1], h]
                    want[2][b[0], h, b[1]], want[3][b[0], h, b[1]] = c.weights[a[0], h, a[1]], c.positions[a[0], h, a[1]]
    for s, w in zip(state, want):
        assert torch.equal(bits(s.t), bits(w))


def test_append_of_malformed_values_stays_inside():
    c, _ = malformed(4, 2, 64, 16, seed=64)
    state = [Guarded(t.shape, t.dtype, 5) for t in (c.k, c.v, c.weights, c.positions)]
    for s, t in zip(state, (c.k, c.v, c.weights, c.positions)):
        s.t.copy_(t)
    rows = torch.tensor([0, -1, 1 << 30, c.total, 3, 1, -(1 << 31)], dtype=torch.int32, device="cuda")
    cache.cache_append(c.k_new, c.v_new, state[0].t, state[1].t, c.table, c.seq_lens, c.cu, rows=rows, weights=state[2].t,
                       positions=state[3].t)
    assert all(s.intact() for s in state)
    # sequence 0 ends at the table's end; the others' slots, pages or rows are not there
    page = int(c.table[0, 4])
    want = [t.clone() for t in (c.k, c.v, c.weights, c.positions)]
    want[0][page, 14], want[1][page, 14], want[2][page, :, 14], want[3][page, :, 14] = c.k_new[0], c.v_new[0], 0.0, 78
    for s, w in zip(state, want):
        assert torch.equal(bits(s.t), bits(w))


# ------------------------------------------------------------ the largest tables and pages
@pytest.mark.parametrize("d", [64, 128])
def test_the_most_sequences(d):
    """2048 sequences, a third without a new token, some empty; 32 heads a key head make full chunks of rows, of
    which fewer fit beside the sequences' table."""
    n = 2048
    lens = [(37 * i) % 90 for i in range(n)]
    new = [0 if i % 3 == 2 else 1 + (i % 5 == 0) * 4 for i in range(n)]
    c = Case(lens, new, 32, 1, d, 16, seed=65, room=8)
    c.weights = torch.nan_to_num(c.weights)
    start = f64(c.weights)
    c.cuda()
    o, lse = cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 5, parents=c.parents)
    check_attention(c, o, lse)
    out = weigh(c, lse, out=torch.zeros_like(c.weights))
    check_weights(c, lse, start, out)
    kept = cache.cache_select(c.weights, c.table, c.seq_lens, 40, 4, c.positions, c.seq_lens)
    assert np.array_equal(kept.cpu().numpy(), ref.select(c, 40, 4, c.seq_lens.cpu()))


@pytest.mark.parametrize("page", [272, 4096, 65536])
def test_large_pages(page):
    d, H, hkv = 64, 4, 2
    c = Case([700, 3, 271], [3, 1, 2], H, hkv, d, page, seed=66, slack=1, room=4)
    start = f64(torch.nan_to_num(c.weights))
    c.cuda()
    o, lse = cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 3, parents=c.parents)
    check_attention(c, o, lse)
    out = weigh(c, lse, out=torch.zeros_like(c.weights))
    check_weights(c, lse, start, out)
    pos = c.seq_lens.clone()
    kept = cache.cache_select(c.weights, c.table, c.seq_lens, 100, 10, c.positions, pos)
    assert np.array_equal(kept.cpu().numpy(), ref.select(c, 100, 10, pos.cpu()))
    cache.cache_compact(kept, c.k, c.v, c.table, c.weights, c.positions)
    c.lens = [100, 3, 100]
    c.seq_lens.clamp_(max=100)
    o, lse = cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 3, parents=c.parents)
    check_attention(c, o, lse)


@pytest.mark.parametrize("width", [20000, 65536, 1 << 20])
def test_selection_under_a_wide_table(width):
    """The table has room for far more than the sequences hold, up to the most a selection takes: the bit map then
    leaves room for fewer keys than the longer sequence has."""
    c = Case([17000, 300], [1, 1], 1, 1, 64, 16, seed=67)
    g = torch.Generator().manual_seed(68)
    c.weights = torch.where(torch.isnan(c.weights), c.weights, torch.round(torch.rand(c.weights.shape, generator=g) * 500))
    c.table = torch.nn.functional.pad(c.table, (0, width // 16 - c.table.shape[1]), value=-1).contiguous()
    c.cuda()
    pos = c.seq_lens.clone()
    for budget in (1, 200, 9000, 16999):
        kept = cache.cache_select(c.weights, c.table, c.seq_lens, budget, min(budget, 30), c.positions, pos)
        assert np.array_equal(kept.cpu().numpy(), ref.select(c, budget, min(budget, 30), pos.cpu()))


# ------------------------------------------------------------ layouts, captures, two at once
def other_layouts(c, kind):
    """(k, v, the tensor they are parts of) of the case in another layout of pages."""
    if kind == "heads first":
        return [t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (c.k, c.v)] + [None]
    if kind == "k and v of a page together":
        both = torch.stack([c.k, c.v], 1)
        return [both[:, 0], both[:, 1], both]
    if kind == "k and v of a head together":
        both = torch.cat([c.k, c.v], -1)
        return [both[..., :c.d], both[..., c.d:], both]
    layers = torch.stack([torch.zeros_like(c.k), c.k, c.v], 2)  # other things between the slots
    return [layers[:, :, 1], layers[:, :, 2], layers]


@pytest.mark.parametrize("kind", ["heads first", "k and v of a page together", "k and v of a head together", "apart"])
@pytest.mark.parametrize("d,hkv", [(64, 2), (128, 1)])
def test_all_operators_on_other_layouts(kind, d, hkv):
    """Pages in strided views: every operator does what it does on dense ones, and nothing between the rows changes."""
    c = Case([100, 33, 300], [4, 1, 2], 4 * hkv, hkv, d, 16, seed=70, room=8).cuda()
    k, v, whole = other_layouts(c, kind)
    results = []
    for kk, vv in ((c.k.clone(), c.v.clone()), (k, v)):
        w, pos = torch.nan_to_num(c.weights), c.positions.clone()
        o, lse = cache.attn_fwd_cache(c.q, c.k_new, c.v_new, kk, vv, c.table, c.seq_lens, c.cu, 4, parents=c.parents)
        after = c.seq_lens + c.cu.diff()
        cache.cache_append(c.k_new, c.v_new, kk, vv, c.table, after, c.cu, weights=w, positions=pos)
        cache.cache_weights(c.q, lse, kk, c.table, after, c.cu, 4, w)
        kept = cache.cache_evict(kk, vv, w, c.table, after, 40, 8, pos, after)
        results.append((o, lse, kk, vv, w, pos, kept))
    for a, b in zip(*results):
        assert torch.equal(bits(a.contiguous()), bits(b.contiguous()))
    if kind == "apart":
        assert (whole[:, :, 0] == 0).all()
    # new tokens as slices of one projection, appended
    packed = torch.cat([c.q, c.k_new, c.v_new], 1)
    a, b = [(t[2].clone(), t[3].clone()) for t in results]
    lens = c.seq_lens + 5
    cache.cache_append(c.k_new, c.v_new, *a, c.table, lens, c.cu)
    cache.cache_append(packed[:, 4 * hkv:5 * hkv], packed[:, 5 * hkv:], *b, c.table, lens, c.cu)
    for x, y in zip(a, b):
        assert torch.equal(bits(x), bits(y.contiguous()))


def test_the_first_calls_of_a_process_are_captured():
    """Nothing of the library has run before: a capture of all operators, replayed."""
    program = textwrap.dedent("""
        import torch
        from cache_reference import Case
        from exact_attention_63_gb300 import cache
        c = Case([900, 40], [900, 40], 8, 1, 64, 16, seed=71, room=8).cuda()
        t = Case([300, 40], [3, 1], 8, 2, 128, 16, seed=72, room=8).cuda()
        c.weights = torch.nan_to_num(c.weights)
        lse = torch.full((8, c.total), 6.0, device="cuda")
        out, k, v = torch.zeros_like(c.weights), c.k.clone(), c.v.clone()
        def step():
            r = cache.attn_fwd_cache(t.q, t.k_new, t.v_new, t.k, t.v, t.table, t.seq_lens, t.cu, 3, parents=t.parents)
            cache.cache_append(c.k_new, c.v_new, k, v, c.table, c.seq_lens, c.cu)
            cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 900, c.weights, out=out)
            kept = cache.cache_select(c.weights, c.table, c.seq_lens, 50, 5)
            cache.cache_compact(kept, k, v, c.table)
            return (*r, kept, k.view(torch.int16), v.view(torch.int16))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        g.replay()
        torch.cuda.synchronize()
        first, got = out.clone(), [x.clone() for x in got]
        k.copy_(c.k)
        v.copy_(c.v)
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(first, out)
        print("fine")
    """)
    tests = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join((os.path.dirname(tests), tests)))
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def test_calls_of_two_threads_at_once():
    """Each thread with its own stream and its own cache."""
    cases = [Case([700, 90], [5, 40], 8, 2, 64, 16, seed=73).cuda(), Case([900], [900], 8, 1, 128, 16, seed=74).cuda()]
    lses = [torch.full((8, c.total), 6.0, device="cuda") for c in cases]
    zeros = [torch.zeros_like(c.weights) for c in cases]

    def work(i):
        c = cases[i]
        r = []
        if i == 0:
            r += cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 40, parents=c.parents)
        r.append(weigh(c, lses[i], out=zeros[i].clone()))
        r.append(cache.cache_select(torch.nan_to_num(c.weights), c.table, c.seq_lens, 30, 5))
        return r

    want = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]

    def loop(i):
        with torch.cuda.stream(streams[i]):
            return [work(i) for _ in range(50)]

    with ThreadPoolExecutor(2) as ex:
        results = [f.result() for f in [ex.submit(loop, i) for i in range(2)]]
    torch.cuda.synchronize()
    for i in range(2):
        for r in results[i]:
            for a, b in zip(r, want[i]):
                used = ~torch.isnan(cases[i].weights) if a.shape == cases[i].weights.shape else slice(None)
                assert torch.equal(a[used], b[used])


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    """Attention and weights of random heads, pages, lengths, trees, bounds, padding, table widths and layouts."""
    rng = random.Random(seed)
    d, hkv, page = rng.choice([64, 128]), rng.choice([1, 2, 3, 8]), rng.choice([16, 32, 48, 64, 128, 272])
    H = hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    n, longest = rng.choice([1, 1, 2, 5, 9, 20]), rng.choice([5, 40, 130, 300, 1000])
    lens = [rng.randint(0, longest) for _ in range(n)]
    new = [rng.choice([0, 1, 1, 2, 5, rng.randint(1, rng.choice([8, 64, 128]))]) for _ in range(n)]
    new[0] = max(new[0], 1)
    c = Case(lens, new, H, hkv, d, page, seed=seed, tree=rng.choice(["random", "chain", "line"]), slack=rng.choice([1, 5]))
    c.weights = torch.nan_to_num(c.weights)
    start, pad = f64(c.weights), rng.choice([0, 3])
    bound = rng.choice([max(new), min(128, max(new) + 7), 128])
    c.table = torch.nn.functional.pad(c.table, (0, rng.choice([0, 3, 500])), value=-1).contiguous()
    c.cuda()
    if rng.random() < 0.4:
        c.k, c.v, _ = other_layouts(c, rng.choice(["heads first", "k and v of a page together", "apart"]))
    padded = [torch.cat([t, torch.full((pad, *t.shape[1:]), float("nan"), device="cuda", dtype=t.dtype)])
              for t in (c.q, c.k_new, c.v_new)]
    parents = None if c.parents is None else torch.cat([c.parents, torch.full((pad,), 5, dtype=torch.int32, device="cuda")])
    o = torch.full((c.total + pad, H, d), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((H, c.total + pad), float("nan"), device="cuda")
    cache.attn_fwd_cache(*padded, c.k, c.v, c.table, c.seq_lens, c.cu, bound, parents=parents, out=o, lse=lse)
    assert (o[c.total:] == 7).all() and torch.isnan(lse[:, c.total:]).all()
    check_attention(c, o[:c.total], lse[:, :c.total])
    outs = [cache.cache_weights(padded[0], lse, c.k, c.table, c.seq_lens, c.cu, bound, c.weights,
                                out=torch.full_like(c.weights, -9.0)) for _ in range(2)]
    check_weights(c, lse[:, :c.total], start, outs[0])
    assert torch.equal(*outs)
