"""Page tables on the GPU against their definition, and a run of the operators around an 8-bit cache."""

from __future__ import annotations

import random

import numpy as np
import pytest
import torch

import fp8_cache_reference as ref8
import oracle
from cache_reference import HALF_BF16, f64
from exact_attention_63_gb300 import attn, cache, rotary
from gpu_common import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    need_gpu()
    assert attn.get_status() == 0
    yield
    assert attn.get_status() == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Tables:
    """The tensors, and lists that follow the definition."""

    def __init__(self, n, width, n_pages, page, seed=0):
        r = random.Random(seed)
        self.table, self.held, self.page = [[-1] * width for _ in range(n)], [0] * n, page
        self.free, self.top = r.sample(range(n_pages), n_pages), n_pages
        self.t, self.h, self.f, self.n = ints(self.table), ints(self.held), ints(self.free), ints([self.top])

    def step(self, lens, new=None, **kw):
        args = {}
        if new is not None:
            args = dict(cu_new=ints([0] + np.cumsum(new).tolist()), total=sum(new))
        missing, slots, positions = cache.cache_pages(ints(lens), self.t, self.h, self.f, self.n, self.page, **args, **kw)
        want, self.top = ref8.resize(self.table, self.held, self.free, self.top, lens, self.page)
        assert missing.tolist() == want
        assert self.n.tolist() == [self.top] and self.h.tolist() == self.held
        assert self.t.tolist() == self.table and self.f.tolist() == self.free
        if new is None:
            assert slots is None and positions is None
            return want
        at, where = [], []
        for s, (n, t) in enumerate(zip(lens, new)):
            for j in range(n - t, n):
                where.append(j)
                at.append(-1 if want[s] or j < 0 else self.table[s][j // self.page] * self.page + j % self.page)
        assert slots.dtype == torch.int64 and slots.tolist() == at and positions.tolist() == where
        return want


def test_grow_shrink_and_end():
    t = Tables(4, 6, 20, 16)
    assert t.step([1, 16, 17, 0], [1, 16, 17, 0]) == [0, 0, 0, 0]
    assert t.step([2, 17, 32, 33], [1, 1, 15, 33]) == [0, 0, 0, 0]
    assert t.step([0, 96, 5, 49]) == [0, 0, 0, 0]
    assert t.step([0, 97, 5, 49], [0, 1, 0, 0])[1] == 1      # wider than the table
    assert t.step([96, 96, 96, 96]) == [0, 0, 5, 2]          # the third and all after it that lack pages wait
    assert t.step([96, 96, 5, 49], [3, 0, 0, 0]) == [0, 0, 0, 0]
    assert t.step([0, 0, 0, 0]) == [0, 0, 0, 0]
    assert sorted(t.f.tolist()) == list(range(20))


@pytest.mark.parametrize("n,width,page", [(1, 700, 16), (33, 40, 16), (257, 9, 48), (2048, 5, 64), (70, 300, 32)])
def test_random_steps(n, width, page):
    r = random.Random(n)
    t = Tables(n, width, n * width * 2 // 3 + 1, page, seed=n)
    most = width * page
    lens = [0] * n
    for i in range(6):
        new = [r.choice([0, 1, 1, 3, most // 2, most + 5 if r.random() < 0.02 else 7]) for _ in range(n)]
        lens = [r.choice([0, a // 2]) if r.random() < 0.2 else min(a + t, most + 3) for a, t in zip(lens, new)]
        missing = t.step(lens, [min(a, t) for a, t in zip(lens, new)] if i % 2 else new)
        lens = [min(a, h * page) if m else a for a, m, h in zip(lens, missing, t.held)]


def test_outputs_streams_and_graphs():
    t = Tables(3, 4, 9, 16)
    lens, cu = ints([16, 20, 3]), ints([0, 16, 20, 23])
    out = [torch.full((3,), 9, dtype=torch.int32, device="cuda"), torch.full((30,), 9, dtype=torch.int64, device="cuda"),
           torch.full((30,), 9, dtype=torch.int32, device="cuda")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cache.cache_pages(lens, t.t, t.h, t.f, t.n, 16, cu, 30, *out, stream=side)
    side.synchronize()
    assert all(a is b for a, b in zip(got, out))
    assert out[1][23:].tolist() == [9] * 7 and out[2].tolist()[:23] == [*range(16), *range(16, 20), *range(3)]
    assert t.h.tolist() == [1, 2, 1] and t.n.tolist() == [5]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cache.cache_pages(lens, t.t, t.h, t.f, t.n, 16, cu, 23)
    lens.copy_(ints([17, 64, 0]))
    graph.replay()
    assert t.h.tolist() == [2, 4, 0] and t.n.tolist() == [3] and got[0].tolist() == [0, 0, 0]
    assert got[2].tolist() == [*range(1, 17), *range(60, 64), *range(-3, 0)] and got[1][20:].tolist() == [-1] * 3
    # many tokens (a second kernel writes the slots) and none
    t = Tables(2, 600, 1300, 16)
    t.step([9000, 9600], [8999, 9600])
    missing, slots, positions = cache.cache_pages(ints([5, 5]), t.t, t.h, t.f, t.n, 16, ints([0, 0, 0]), 0)
    assert slots.shape == positions.shape == (0,)


def test_counts_out_of_range():
    """Garbage in the counts: nothing outside the tensors is touched."""
    t = Tables(3, 4, 9, 16)
    for held, top, lens in (([99, -5, 2], 7, [1, 50, 64]), ([4, 4, 4], 9, [0, 0, 0]), ([0, 0, 0], 1 << 30, [64, 64, 64]),
                            ([0, 0, 0], -4, [64, 1, -7]), ([1, 1, 1], 3, [2 ** 31 - 1, 2 ** 31 - 1, -(2 ** 31)])):
        free = torch.arange(9 + 8, dtype=torch.int32, device="cuda")
        cache.cache_pages(ints(lens), t.t, ints(held), free[4:13], ints([top]), 16, ints([5, 900, -3, 2]), 30)
        assert free[:4].tolist() == [0, 1, 2, 3] and free[13:].tolist() == [13, 14, 15, 16]


def test_refusals():
    t = Tables(3, 4, 9, 16)
    ok = dict(seq_lens=ints([1, 1, 1]), block_table=t.t, n_blocks=t.h, free_pages=t.f, n_free=t.n, page_size=16)
    cache.cache_pages(**ok)
    cu = ints([0, 1, 2, 3])
    for kw in (dict(seq_lens=ints([1])), dict(seq_lens=None), dict(block_table=t.t.long()), dict(block_table=t.t[:, ::2]),
               dict(block_table=t.t.cpu()), dict(n_blocks=ints([1, 1])), dict(free_pages=t.f[None]), dict(n_free=ints([1, 1])),
               dict(cu_new=ints([0, 1]), total=1), dict(total=3), dict(cu_new=cu, total=-1), dict(missing=ints([1])),
               dict(cu_new=cu, total=3, slots=ints([1, 1, 1])), dict(cu_new=cu, total=3, positions=ints([1])), dict(slots=ints([1]).long())):
        with pytest.raises(ValueError):
            cache.cache_pages(**{**ok, **kw})
    for page in (0, 8, 24, 65552):
        with pytest.raises(attn.AttnError):
            cache.cache_pages(**{**ok, "page_size": page})


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_and_steps(d):
    """Two requests as a server runs them: pages for the prompts, rotary positions, attention over the prompt, its
    rows into the 8-bit cache; a second piece of one prompt over the gathered rows; then steps of a drafted chain,
    of which some tokens are taken.  Every attention against float64 over what the cache stands for."""
    H, hkv, page, G = 8, 2, 16, 4
    g = torch.Generator().manual_seed(d)
    rnd = lambda rows, heads: torch.randn((rows, heads, d), generator=g).bfloat16().cuda()  # noqa: E731
    t = Tables(2, 40, 70, page, seed=d)
    codes = [torch.full((70, page, hkv, d), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((70, hkv, 1), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pages = (*codes, *scales)
    freq = rotary.rotary_frequencies(d, scaling="by_parts", factor=4.0).cuda()

    def room(lens, new):
        cu = ints([0] + np.cumsum(new).tolist())
        missing, _, positions = cache.cache_pages(ints(lens), t.t, t.h, t.f, t.n, page, cu, sum(new))
        assert missing.tolist() == [0, 0]
        q, k = rotary.rotary_fwd(rnd(sum(new), H), rnd(sum(new), hkv), positions, freq, magnitude=1.1)
        return cu, q, k, rnd(sum(new), hkv)

    def against(o, q, K, V, rows, offset):
        for h in range(H):
            one = lambda x: x[:, h // G][None, :, None].cpu()  # noqa: E731
            O, _ = oracle.attention_forward(q[rows][None, :, h:h + 1].cpu(), one(K), one(V), d ** -0.5, True, causal_offset=offset)
            err = np.abs(f64(o[rows, h]) - O[0, :, 0]) - (1e-2 + 1e-2 * np.abs(O[0, :, 0]))
            assert err.max() <= 0

    def held(s, n):
        at = t.t[s].long()[torch.arange(n, device="cuda") // page]
        place = torch.arange(n) % page
        return [torch.from_numpy(ref8.values(c.cpu().numpy(), x.cpu().numpy()))[at.cpu(), place].bfloat16().cuda()
                for c, x in zip(codes, scales)]

    lens, new = [130, 301], [130, 301]
    cu, q, k, v = room(lens, new)
    o, _ = attn.attn_fwd_varlen(q, k, v, cu, cu, 301, causal=True)
    cache.cache_append_fp8(k, v, *pages, t.t, ints(lens), cu)
    for s in range(2):
        r = slice(int(cu[s]), int(cu[s + 1]))
        against(o, q, k[r], v[r], r, 0)
        for x, y in zip(held(s, lens[s]), (k[r], v[r])):
            # a code is off by 2^-4 of its value, or half of its smallest step in units of a scale of at most
            # the block's largest value / 224
            assert (np.abs(f64(x) - f64(y)) <= 2.0 ** -4 * np.abs(f64(y)) + 2.0 ** -10 * np.abs(f64(y)).max() / 224).all()
    # the second piece of request 0: longer than a draft
    before, lens, new = lens, [130 + 150, 301], [150, 0]
    cu, q, k, v = room(lens, new)
    cu_ctx = ints([0, 130, 130])
    K, V = cache.cache_gather_fp8(*pages, t.t, ints(before), cu_ctx, 130)
    cu_k = ints([0, 280, 280])
    o, _ = attn.attn_fwd_varlen(q, torch.cat([K, k]), torch.cat([V, v]), cu, cu_k, 150, causal=True, causal_align="bottom-right")
    want = held(0, 130)
    assert torch.equal(K, want[0]) and torch.equal(V, want[1])
    against(o, q, torch.cat([K, k]), torch.cat([V, v]), slice(0, 150), 130)
    cache.cache_append_fp8(k, v, *pages, t.t, ints(lens), cu)
    # steps: three drafted tokens each, of which one and two are taken
    for step in range(4):
        drafted = [a + 3 for a in lens]
        cu, q, k, v = room(drafted, [3, 3])
        o, _ = cache.attn_fwd_cache_fp8(q, k, v, *pages, t.t, ints(lens), cu, 3)
        for s in range(2):
            K, V = held(s, lens[s])
            r = slice(3 * s, 3 * s + 3)
            against(o, q, torch.cat([K, k[r]]), torch.cat([V, v[r]]), r, lens[s])
        lens = [lens[0] + 1, lens[1] + 2]
        missing, _, _ = cache.cache_pages(ints(lens), t.t, t.h, t.f, t.n, page)  # what the rejected ones held goes back
        cache.cache_append_fp8(k, v, *pages, t.t, ints(lens), ints([0, 1, 3]), rows=ints([0, 3, 4]))
    assert t.h.tolist() == [-(-a // page) for a in lens]
    cache.cache_pages(ints([0, 0]), t.t, t.h, t.f, t.n, page)
    assert sorted(t.f.tolist()) == list(range(70)) and t.n.tolist() == [70]
