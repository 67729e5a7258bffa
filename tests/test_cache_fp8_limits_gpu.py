"""The 8-bit cache's operators at the edges of their contract: tables, lengths and offsets out of range between guard
bands, a workspace of exactly its size, far pages under every kernel, and how precise P is where rows are few."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import cache_reference as ref
import fp8_cache_reference as ref8
from cache_reference import HALF_BF16, f64
from exact_attention_63_gb300 import attn, cache
from fp8_cache_reference import Fp8Case
from gpu_common import need_gpu

HALF_F16 = 2.0 ** -11


@pytest.fixture
def gpu():
    need_gpu()
    assert attn.get_status() == 0
    yield
    assert attn.get_status() == 0


class Guarded:
    """A tensor between margins of 4 KB, all of them filled with a pattern that has to stay."""

    def __init__(self, shape, dtype, like=None, align=256):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.n, self.margin = n, 4096
        self.raw = torch.full((n + 2 * self.margin + align,), 0xA5, dtype=torch.uint8, device="cuda")
        self.at = -(-(self.raw.data_ptr() + self.margin) // align) * align - self.raw.data_ptr()
        self.t = self.raw[self.at:self.at + n].view(dtype).view(shape)
        if like is not None:
            self.t.copy_(like)

    def check(self):
        assert bool((self.raw[:self.at] == 0xA5).all()) and bool((self.raw[self.at + self.n:] == 0xA5).all())


def guarded_cache(c):
    """c's codes and scales inside guard bands; the four Guarded."""
    out = []
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        x = getattr(c, name)
        g = Guarded(x.shape, torch.uint8, x)
        setattr(c, name, g.t)
        out.append(g)
    return out


# the new tokens of a sequence: tiles of 8, 16 (d = 64: 32) rows, one row tile of the converting kernel, two of them
NEW = [1, 9, 40, 100]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("offsets", [None, [0, 999, -3, 4], [7, 2, 5, 1 << 30], [-(1 << 31), 3, 3, 3]], ids=["cu", "behind", "back", "before"])
def test_attention_of_malformed_calls_stays_inside(gpu, new, d, offsets):
    """Pages and lengths out of range, and offsets out of range or order: nothing outside o, lse and the workspace
    is written, rows of no sequence stay, and a sequence that is not concerned is right."""
    c = Fp8Case([300, 90, 200], [new, min(new, 2), new], 4, 2, d, 16, seed=12).cuda()
    O, L, A = ref.attention(c)
    eps = ref.score_bound(c)
    tables = guarded_cache(c)
    before = [g.t.clone() for g in tables]
    c.table[0, 3], c.table[1, 0] = 1 << 30, -5
    c.seq_lens.copy_(torch.tensor([1 << 30, -7, 200]))
    cu = c.cu if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    o, lse = Guarded((c.total, 4, d), torch.bfloat16), Guarded((4, c.total), torch.float32)
    ws = Guarded((cache.workspace_size_fp8(4, 2, new, d),), torch.uint8)
    was = o.t.clone()
    cache.attn_fwd_cache_fp8(c.q, c.k_new, c.v_new, *c.pages(), c.table, c.seq_lens, cu, new, parents=c.parents, out=o.t, lse=lse.t,
                             workspace=ws.t)
    torch.cuda.synchronize()
    for g in (o, lse, ws, *tables):
        g.check()
    for g, x in zip(tables, before):
        assert torch.equal(g.t, x)
    if offsets is None:
        r = slice(int(c.cu[2]), int(c.cu[3]))
        tol = HALF_BF16 * (A + np.abs(O)) * (1 + HALF_BF16) + (4 * eps + 2.0 ** -20) * A + 400 * 2.0 ** -32 * 10
        assert (np.abs(f64(o.t) - O) <= tol)[r].all()
        assert (np.abs(f64(lse.t) - L) <= 2 * eps + 2.0 ** -20 * (1 + np.abs(L)))[:, r].all()
    else:
        cl = np.clip(np.array(offsets, np.int64), 0, c.total)
        owned = np.zeros(c.total, bool)
        for a, z in zip(cl[:-1], cl[1:]):
            owned[a:min(max(a, z), a + new)] = True
        rest = torch.from_numpy(~owned).cuda()
        assert torch.equal(o.t[rest].view(torch.int16), was[rest].view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_append_to_malformed_tables_is_that_to_the_clamped_ones(gpu, hkv, d):
    """Pages out of range are not written, lengths are clamped to the table: codes and scales by the definition, bit
    for bit, those of every other page among them, and nothing beside them."""
    new = [60, 40, 3, 50]
    c = Fp8Case([30, 20, 40, 0], new, hkv, hkv, d, 16, seed=13, room=60).cuda()
    blocks = c.table.shape[1]
    c.table[0, 3], c.table[1, 2], c.table[3, :] = c.n_pages, -(1 << 31), 1 << 30
    c.table[2, :3] = torch.tensor([-1, 2 ** 31 - 1, int(c.table[2, 2])])
    lens = [90, 1 << 30, 43, 50]
    clamped = [min(x, 16 * blocks) for x in lens]
    tables = guarded_cache(c)
    want = []
    for name in ("k", "v"):
        codes, scales = getattr(c, name + "_codes").cpu().numpy().copy(), getattr(c, name + "_scales").cpu().numpy().copy()
        ref8.append(codes, scales, c.table.cpu().numpy(), clamped, c.cu.tolist(), f64(getattr(c, name + "_new")))
        want.append((codes, scales))
    start = [g.t.clone() for g in tables]
    cache.cache_append_fp8(c.k_new, c.v_new, *c.pages(), c.table, torch.tensor(lens, dtype=torch.int32, device="cuda"), c.cu)
    torch.cuda.synchronize()
    for g in tables:
        g.check()
    got = [g.t.cpu().numpy() for g in tables]
    for i in range(2):
        assert np.array_equal(got[i], want[i][0]) and np.array_equal(got[2 + i], want[i][1])
    assert not torch.equal(start[0], tables[0].t)  # (some of it was written)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("offsets", [[0, 999, -3, 4], [7, 2, 5, 1 << 30], [-(1 << 31), 3, 3, 3], [5, 5, 90, 60]], ids=["behind", "back", "before", "late"])
def test_append_of_malformed_offsets_stays_in_the_tables_pages(gpu, offsets, rows):
    c = Fp8Case([30, 20, 40], [30, 30, 30], 3, 3, 64, 32, seed=14, room=70, slack=6).cuda()
    tables = guarded_cache(c)
    before = [g.t.clone() for g in tables]
    lens = torch.tensor([60, 2 ** 31 - 1, -(1 << 31)], dtype=torch.int32, device="cuda")
    which = torch.arange(-4, 86, dtype=torch.int32, device="cuda") if rows else None
    cache.cache_append_fp8(c.k_new, c.v_new, *c.pages(), c.table, lens, torch.tensor(offsets, dtype=torch.int32, device="cuda"), rows=which)
    torch.cuda.synchronize()
    used = c.table.unique()
    rest = torch.ones(c.n_pages, dtype=torch.bool, device="cuda")
    rest[used[used >= 0].long()] = False
    assert int(rest.sum()) >= 6
    for g, x in zip(tables, before):
        g.check()
        assert torch.equal(g.t[rest], x[rest])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_gather_of_malformed_calls_stays_inside(gpu, hkv, d):
    c = Fp8Case([90, 40, 33], [1, 1, 1], hkv, hkv, d, 16, seed=15).cuda()
    cap = 16 * c.table.shape[1]
    tables = guarded_cache(c)
    kept = [g.t.clone() for g in tables]
    table = c.table.clone()
    c.table[0, 3], c.table[1, 0] = 1 << 30, -(1 << 31)
    for lens, offsets in (([90, 40, 33], [0, 90, 130, 163]), ([1 << 30, -7, 33], [0, 90, 130, 163]), ([90, 40, 33], [5, 999, -3, 40]),
                          ([90, 40, 33], [1 << 30, 2, 1, -(1 << 31)])):
        total = 170
        k, v = Guarded((total, hkv, d), torch.bfloat16), Guarded((total, hkv, d), torch.bfloat16)
        was = k.t.clone()
        cache.cache_gather_fp8(*c.pages(), c.table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               torch.tensor(offsets, dtype=torch.int32, device="cuda"), total, k.t, v.t)
        torch.cuda.synchronize()
        for g in (k, v, *tables):
            g.check()
        for g, x in zip(tables, kept):
            assert torch.equal(g.t, x)
        if offsets[1] != 90:
            continue
        for s, n in enumerate(lens):  # rows on the pages that are in range
            n, a, z = min(max(n, 0), cap), offsets[s], offsets[s + 1]
            for i in range(a, z):
                j = n - z + i
                for got, x in ((k, c.k), (v, c.v)):
                    if j < 0:
                        assert torch.equal(got.t[i].view(torch.int16), was[i].view(torch.int16))
                    elif table[s, j // 16] >= 0 and table[s, j // 16] == c.table[s, j // 16] and j < c.lens[s]:
                        assert torch.equal(got.t[i], x[int(table[s, j // 16]), j % 16])
        assert torch.equal(k.t[163:].view(torch.int16), was[163:].view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("new", NEW)
def test_attention_over_pages_beyond_32_bits(gpu, new):
    """Every kernel reads the pages that lie behind 4 GB as it reads the same ones near."""
    n_pages, page, hkv, d = 4200, 1024, 8, 128  # 4.4 GB of codes
    c = Fp8Case([0, 0], [new, new], 32, hkv, d, 16, seed=17, room=300).cuda()
    g = torch.Generator().manual_seed(18)
    prompt = [torch.randn((500, hkv, d), generator=g).bfloat16().cuda() for _ in range(2)]
    lens = torch.tensor([230, 270], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 230, 500], dtype=torch.int32, device="cuda")
    cache.cache_append_fp8(*prompt, *c.pages(), c.table, lens, cu)
    near = cache.attn_fwd_cache_fp8(c.q, c.k_new, c.v_new, *c.pages(), c.table, lens, c.cu, new, parents=c.parents)
    k, v = (torch.zeros((n_pages, page, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((n_pages, hkv, page // 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.tensor([[n_pages - 1], [n_pages - 3]], dtype=torch.int32, device="cuda")
    cache.cache_append_fp8(*prompt, k, v, ks, vs, table, lens, cu)
    far = cache.attn_fwd_cache_fp8(c.q, c.k_new, c.v_new, k, v, ks, vs, table, lens, c.cu, new, parents=c.parents)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
    assert torch.isfinite(near[0].float()).all()


# ------------------------------------------------------------------ how precise P is with few rows


def nearly_cancelling(new, d):
    """Sequences of two keys whose values are opposite and whose weights nearly equal: what is left of their sum
    shows how P was rounded, far above the rounding of the result.  A token's own key has next to no weight."""
    c = Fp8Case([2] * 40, [new] * 40, 8, 8, d, 16, seed=30, tree="roots")
    table = c.table.numpy()
    codes = c.v_codes.numpy()
    for s in range(40):
        codes[table[s, 0], 1] = codes[table[s, 0], 0] ^ 128
    c.v = torch.from_numpy(ref8.values(codes, c.v_scales.numpy())).bfloat16()
    c.k_new = (c.q.float() * -100).bfloat16()
    c.scale = 0.05 / d ** 0.5
    return c


def parts(c):
    """float64: O and Σ p|v| over the cached keys, Σ p|v| over the new ones, and the cached keys' weights and values."""
    q, kn, vn, k, v = (f64(x) for x in (c.q, c.k_new, c.v_new, c.k, c.v))
    table, out = c.table.cpu().numpy(), [np.zeros((c.total, c.H, c.d)) for _ in range(3)]
    P, V = np.zeros((c.total, c.H, 2)), np.zeros((c.total, c.H, 2, c.d))
    for i in range(c.total):
        s = i // c.new[0]
        for h in range(c.H):
            z = np.append(k[table[s, 0], :2, h] @ q[i, h], kn[i, h] @ q[i, h]) * c.scale
            p = np.exp(z - z.max())
            p /= p.sum()
            vals = v[table[s, 0], :2, h]
            out[0][i, h] = p[:2] @ vals + p[2] * vn[i, h]
            out[1][i, h], out[2][i, h] = p[:2] @ np.abs(vals), p[2] * np.abs(vn[i, h])
            P[i, h], V[i, h] = p[:2], vals
    return (*out, P, V)


def bound(c, O, cached, own):
    """P of cached keys rounded to f16 and of new ones to bf16, the result once; scores off by the fp32 sum of d
    products (the cached keys', the others have no weight to speak of); 2^-32 below f16's range."""
    big = np.linalg.norm(f64(c.q), axis=-1).max() * np.linalg.norm(np.nan_to_num(f64(c.k)), axis=-1).max() * c.scale
    eps = (c.d + 8) * ref.HALF_F32 * big + 2.0 ** -20
    return HALF_BF16 * np.abs(O) * (1 + HALF_BF16) + (HALF_F16 * cached + HALF_BF16 * own) * (1 + HALF_BF16) + \
        (4 * eps + 2.0 ** -20) * cached + 3 * 2.0 ** -32 * np.nan_to_num(f64(c.v)).max()


FEW = [(64, 1), (64, 12), (64, 30), (128, 1), (128, 12)]


@pytest.mark.parametrize("d,new", FEW)
def test_the_bound_on_p_tells_f16_from_bf16(d, new):
    """The oracle with P in f16 passes, with P in bf16 it does not (P in units where the larger is 2^7)."""
    c = nearly_cancelling(new, d)
    O, cached, own, P, V = parts(c)
    tol = bound(c, O, cached, own)
    units = 128.0 / P.max(-1, keepdims=True)
    for dtype, passes in ((torch.float16, True), (torch.bfloat16, False)):
        rounded = torch.from_numpy(P * units).float().to(dtype).double().numpy() / units
        got = torch.from_numpy(O + ((rounded - P)[..., None] * V).sum(2)).bfloat16()
        assert bool((np.abs(f64(got) - O) <= tol).all()) is passes


@pytest.mark.gpu
@pytest.mark.parametrize("d,new", FEW)
def test_p_is_f16_where_rows_are_few(gpu, d, new):
    c = nearly_cancelling(new, d)
    O, cached, own, _, _ = parts(c)
    tol = bound(c, O, cached, own)
    c.cuda()
    o, _ = cache.attn_fwd_cache_fp8(c.q, c.k_new, c.v_new, *c.pages(), c.table, c.seq_lens, c.cu, new, parents=c.parents, scale=c.scale)
    assert (np.abs(f64(o) - O) <= tol).all()
