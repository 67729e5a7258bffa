"""The 8-bit cache's operators, the page tables and the rotary positions refuse bad arguments before any
launch (no GPU needed)."""

from __future__ import annotations

import ctypes

import pytest
import torch

from exact_attention_63_gb300 import attn, cache, rotary
from test_cache_abi import A, L, a_cache, tokens  # noqa: F401

NULL, SHAPE, DIM, SCALE, ALIGN, ARCH, OPTION, WORKSPACE, LAYOUT, CACHE = -1, -2, -3, -4, -5, -6, -9, -10, -12, -13


def calls(L, c, x, ks=A, vs=A, scale=0.125, o=A, lse=A, ws=A, ws_bytes=1 << 40, opts=None, rows=None, n_rows=0, cu=A, total=5,  # noqa: F811
          k_out=A, v_out=A):
    cp = None if c is None else ctypes.byref(c)
    xp = None if x is None else ctypes.byref(x)
    op = None if opts is None else ctypes.byref(opts)
    return {
        "attend": lambda: L.attn_fwd_cache_fp8(cp, ks, vs, xp, A, scale, o, lse, ws, ws_bytes, op, None),
        "append": lambda: L.attn_cache_append_fp8(cp, ks, vs, xp, rows, n_rows, None),
        "gather": lambda: L.attn_cache_gather_fp8(cp, ks, vs, cu, total, k_out, v_out, None),
    }


ALL = ("attend", "append", "gather")


@pytest.mark.parametrize("field,value,expect", [
    ("block_table", None, NULL), ("seq_lens", None, NULL), ("k", None, NULL), ("v", None, NULL), ("struct_size", 8, CACHE),
    ("page_size", 24, CACHE), ("page_size", 0, CACHE), ("n_seq", 2049, CACHE), ("n_pages", 0, SHAPE), ("max_blocks", 0, SHAPE),
    ("max_blocks", 1 << 27, CACHE), ("num_kv_heads", 0, SHAPE), ("d", 96, DIM), ("k", A + 8, ALIGN), ("v", A + 8, ALIGN),
    ("k_strides", (2048, 128, 72), CACHE), ("v_strides", (2048, 0, 64), CACHE), ("k_strides", (1 << 38, 128, 64), CACHE),
    ("block_table", A + 2, ALIGN), ("seq_lens", A + 1, ALIGN),
])
def test_cache_fields(L, field, value, expect):  # noqa: F811
    run = calls(L, a_cache(**{field: value}), tokens())
    for op in ALL:
        assert run[op]() == expect, op


@pytest.mark.parametrize("kw,expect,ops", [
    (dict(c=None), NULL, ALL), (dict(x=None), NULL, ("attend", "append")), (dict(ks=None), NULL, ALL), (dict(vs=None), NULL, ALL),
    (dict(o=None), NULL, ("attend",)), (dict(lse=None), NULL, ("attend",)), (dict(cu=None), NULL, ("gather",)),
    (dict(k_out=None), NULL, ("gather",)), (dict(v_out=None), NULL, ("gather",)), (dict(total=0), SHAPE, ("gather",)),
    (dict(total=(1 << 30) + 1), SHAPE, ("gather",)), (dict(k_out=A + 8), ALIGN, ("gather",)), (dict(cu=A + 2), ALIGN, ("gather",)),
    (dict(scale=0.0), SCALE, ("attend",)), (dict(scale=float("inf")), SCALE, ("attend",)), (dict(o=A + 8), ALIGN, ("attend",)),
    (dict(lse=A + 2), ALIGN, ("attend",)), (dict(ws=None), WORKSPACE, ("attend",)), (dict(ws=A + 16), WORKSPACE, ("attend",)),
    (dict(ws_bytes=1000), WORKSPACE, ("attend",)), (dict(rows=A, n_rows=0), SHAPE, ("append",)),
    (dict(rows=A + 2, n_rows=1), ALIGN, ("append",)),
    (dict(opts=attn.make_options(rescale_threshold=1.0)), OPTION, ("attend",)),
    (dict(opts=attn.make_options(test_flags=2)), OPTION, ("attend",)),
])
def test_arguments(L, kw, expect, ops):  # noqa: F811
    run = calls(L, kw.pop("c", a_cache()), kw.pop("x", tokens()), **kw)
    for op in ops:
        assert run[op]() == expect, op


@pytest.mark.parametrize("field,value,expect,ops", [
    ("cu_seqlens", None, NULL, ("attend", "append")), ("q", None, NULL, ("attend",)), ("k", None, NULL, ("attend", "append")),
    ("total", 0, SHAPE, ("attend", "append")), ("total", (1 << 30) + 1, SHAPE, ("append",)), ("max_seqlen", 129, SHAPE, ("attend",)),
    ("H", 5, CACHE, ("attend",)), ("q", A + 8, ALIGN, ("attend",)), ("v", A + 4, ALIGN, ("attend", "append")),
    ("q_strides", (256, 60), CACHE, ("attend",)), ("k_strides", (0, 64), CACHE, ("attend", "append")),
])
def test_token_fields(L, field, value, expect, ops):  # noqa: F811
    run = calls(L, a_cache(), tokens(**{field: value}))
    for op in ops:
        assert run[op]() == expect, op


def test_valid_calls_need_a_device(L):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("fake addresses")
    for op, run in calls(L, a_cache(), tokens()).items():
        assert run() == ARCH, op
    assert pages(L) == ARCH and turn(L) == ARCH


def test_workspace_sizes(L):  # noqa: F811
    size = cache.workspace_size_fp8
    assert size(8, 2, 0, 64) == size(8, 2, 129, 64) == size(8, 3, 1, 64) == size(8, 2, 1, 96) == size(258, 2, 1, 64) == 0
    for H, hkv in ((1, 1), (8, 2), (32, 8), (128, 1)):
        for d in (64, 128):
            sizes = [size(H, hkv, n, d) for n in range(1, 129)]
            assert sizes[0] > 0 and sizes == sorted(sizes)  # one for the largest serves the smaller


def pages(L, lens=A, missing=A, cu=A, total=4, slots=A, positions=A, null=False, **kw):  # noqa: F811
    t = cache.Pages()
    t.struct_size = ctypes.sizeof(cache.Pages)
    t.block_table = t.n_blocks = t.free_pages = t.n_free = A
    t.n_seq, t.max_blocks, t.n_pages, t.page_size = 3, 4, 9, 16
    for k, v in kw.items():
        setattr(t, k, v)
    return L.attn_cache_pages(None if null else ctypes.byref(t), lens, missing, cu, total, slots, positions, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(null=True), NULL), (dict(lens=None), NULL), (dict(missing=None), NULL), (dict(slots=None), NULL), (dict(positions=None), NULL),
    (dict(block_table=None), NULL), (dict(n_blocks=None), NULL), (dict(free_pages=None), NULL), (dict(n_free=None), NULL),
    (dict(struct_size=8), CACHE), (dict(n_seq=0), SHAPE), (dict(n_seq=2049), CACHE), (dict(max_blocks=0), SHAPE), (dict(n_pages=0), SHAPE),
    (dict(page_size=8), CACHE), (dict(page_size=24), CACHE), (dict(page_size=65552), CACHE), (dict(total=-1), SHAPE),
    (dict(total=(1 << 30) + 1), SHAPE), (dict(max_blocks=1 << 27), CACHE), (dict(n_seq=2048, max_blocks=1 << 20), SHAPE),
    (dict(lens=A + 2), ALIGN), (dict(slots=A + 4), ALIGN), (dict(cu=A + 1), ALIGN), (dict(n_free=A + 2), ALIGN),
])
def test_pages(L, kw, expect):  # noqa: F811
    assert pages(L, **kw) == expect


def turn(L, q=True, k=True, batch=2, rows=5, d=64, positions=A, apart=5, freq=A, part=64, magnitude=1.0, **kw):  # noqa: F811
    sides = []
    for there in (q, k):
        r = rotary.Rows()
        r.struct_size, r.x, r.y, r.heads = ctypes.sizeof(rotary.Rows), A, A, 4
        for name, v in kw.items():
            if name.endswith("strides"):
                getattr(r, name)[:] = v
            else:
                setattr(r, name, v)
        sides.append(ctypes.byref(r) if there else None)
    return L.attn_rotary(*sides, batch, rows, d, positions, apart, freq, part, 0, magnitude, 0, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=False), NULL), (dict(freq=None), NULL), (dict(x=None), NULL), (dict(y=None), NULL), (dict(struct_size=8), LAYOUT),
    (dict(batch=0), SHAPE), (dict(rows=0), SHAPE), (dict(batch=1 << 20, rows=1 << 20), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=65537), SHAPE), (dict(d=96), DIM), (dict(d=256), DIM), (dict(part=0), LAYOUT), (dict(part=3), LAYOUT),
    (dict(part=66), LAYOUT), (dict(apart=-1), LAYOUT), (dict(magnitude=float("nan")), SCALE), (dict(x=A + 8), ALIGN),
    (dict(y=A + 2), ALIGN), (dict(positions=A + 2), ALIGN), (dict(freq=A + 4), ALIGN), (dict(x_strides=(2048, 256, 60)), LAYOUT),
    (dict(y_strides=(0, 256, 64)), LAYOUT), (dict(x_strides=(2048, -256, 64)), LAYOUT), (dict(y_strides=(1 << 38, 256, 64)), LAYOUT),
])
def test_rotary(L, kw, expect):  # noqa: F811
    assert turn(L, **kw) == expect


def test_frequencies():
    f = rotary.rotary_frequencies(64)
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1.0 and abs(f[31] - 10000.0 ** (-62 / 64)) < 1e-15
    assert torch.equal(rotary.rotary_frequencies(64, scaling="linear", factor=4.0), f / 4.0)
    g = rotary.rotary_frequencies(64, scaling="base", factor=4.0)
    assert g[0] == 1.0 and abs(float(g[31] * 4.0 / f[31]) - 1.0) < 1e-12
    h = rotary.rotary_frequencies(64, scaling="by_parts", factor=4.0, original_length=4096)
    turns = 4096 * f / (2 * torch.pi)
    assert torch.equal(h[turns > 40], f[turns > 40]) and torch.allclose(h[turns < 0.7], f[turns < 0.7] / 4.0, rtol=1e-15)
    assert (h <= f).all() and (h >= f / 4.0 * (1 - 1e-15)).all() and (h[1:] < h[:-1]).all()
    assert rotary.rotary_magnitude(1.0) == 1.0 and rotary.rotary_magnitude(8.0) > 1.2
    for kw in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, base=1.0),
               dict(rotary_dim=8, factor=0.0), dict(rotary_dim=2, scaling="base"), dict(rotary_dim=8, scaling="by_parts", turns=(1.0, 32.0))):
        with pytest.raises(ValueError):
            rotary.rotary_frequencies(**kw)


def test_tensors_that_are_not_on_a_gpu_are_refused():
    x = torch.zeros(4, 2, 64).bfloat16()
    t = torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError):
        rotary.rotary_fwd(x, x, None, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        cache.cache_pages(t[0], t, t[0], t[0], t[0], 16)
    codes, scales = torch.zeros((1, 16, 2, 64), dtype=torch.uint8), torch.zeros((1, 2, 1), dtype=torch.uint8)
    with pytest.raises(ValueError):
        cache.attn_fwd_cache_fp8(x, x, x, codes, codes, scales, scales, t, t[0], t[0], 1)
    with pytest.raises(ValueError):
        cache.cache_append_fp8(x, x, codes, codes, scales, scales, t, t[0], t[0])
    with pytest.raises(ValueError):
        cache.cache_gather_fp8(codes, codes, scales, scales, t, t[0], t[0], 1)
