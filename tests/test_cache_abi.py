"""The cache operators refuse bad arguments before any launch (no GPU needed)."""

from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

from exact_attention_63_gb300 import attn, cache

A = 0x10000  # a fake, 16-byte aligned "device" address: never dereferenced
NULL, SHAPE, DIM, SCALE, ALIGN, ARCH, OPTION, WORKSPACE, CACHE = -1, -2, -3, -4, -5, -6, -9, -10, -13
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "attn_gb300.h")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(attn._LIB_PATH):
        from exact_attention_63_gb300 import build

        build.build()
    return attn.lib()


def a_cache(**kw):
    c = cache.Cache()
    c.struct_size = ctypes.sizeof(cache.Cache)
    for name in ("k", "v", "weights", "positions", "block_table", "seq_lens"):
        setattr(c, name, A)
    c.n_pages, c.page_size, c.max_blocks, c.n_seq, c.num_kv_heads, c.d = 20, 16, 10, 2, 2, 64
    for k, v in kw.items():
        if k.endswith("_strides"):
            getattr(c, k)[:] = v
        else:
            setattr(c, k, v)
    return c


def tokens(**kw):
    x = cache.NewTokens()
    x.struct_size = ctypes.sizeof(cache.NewTokens)
    x.q = x.k = x.v = x.cu_seqlens = A
    x.total, x.max_seqlen, x.H = 6, 3, 4
    for k, v in kw.items():
        if k.endswith("_strides"):
            getattr(x, k)[:] = v
        else:
            setattr(x, k, v)
    return x


def calls(L, c, x, scale=0.125, o=A, lse=A, ws=A, ws_bytes=1 << 40, opts=None, kept=A, budget=8, recent=2, seq_pos=A,
          rows=None, n_rows=0, parents=A, out=A):
    """Status of each entry point for these arguments."""
    cp = None if c is None else ctypes.byref(c)
    xp = None if x is None else ctypes.byref(x)
    op = None if opts is None else ctypes.byref(opts)
    return {
        "attend": lambda: L.attn_fwd_cache(cp, xp, parents, scale, o, lse, ws, ws_bytes, op, None),
        "append": lambda: L.attn_cache_append(cp, xp, rows, n_rows, seq_pos, None),
        "weigh": lambda: L.attn_cache_weights(cp, xp, lse, scale, out, op, None),
        "select": lambda: L.attn_cache_select(cp, seq_pos, budget, recent, kept, None),
        "compact": lambda: L.attn_cache_compact(cp, kept, budget, None),
    }


ALL = ("attend", "append", "weigh", "select", "compact")
PAGED = ("attend", "append", "weigh", "compact")   # those that read k


@pytest.mark.parametrize("field,value,expect,ops", [
    ("block_table", None, NULL, ALL), ("seq_lens", None, NULL, ("attend", "append", "weigh", "select")),
    ("k", None, NULL, PAGED), ("v", None, NULL, ("attend", "append", "compact")),
    ("weights", None, NULL, ("select",)),
    ("struct_size", 8, CACHE, ALL), ("page_size", 0, CACHE, ALL), ("page_size", 24, CACHE, ALL),
    ("page_size", 65552, CACHE, ALL), ("n_seq", 0, SHAPE, ALL), ("n_seq", 2049, CACHE, ALL),
    ("n_pages", 0, SHAPE, ALL), ("max_blocks", 0, SHAPE, ALL), ("max_blocks", 1 << 27, CACHE, ALL),
    ("num_kv_heads", 0, SHAPE, ALL), ("num_kv_heads", 3, CACHE, ("attend", "weigh")),
    ("d", 96, DIM, PAGED), ("k", A + 8, ALIGN, PAGED), ("v", A + 8, ALIGN, ("attend", "append", "compact")),
    ("block_table", A + 2, ALIGN, ALL), ("seq_lens", A + 1, ALIGN, ALL), ("weights", A + 4, ALIGN, ALL),
    ("positions", A + 8, ALIGN, ALL),
    ("k_strides", (2048, 128, 60), CACHE, PAGED), ("k_strides", (2048, 0, 64), CACHE, PAGED),
    ("v_strides", (-2048, 128, 64), CACHE, ("attend", "append", "compact")),
    ("k_strides", (1 << 38, 128, 64), CACHE, PAGED),
    ("max_blocks", (1 << 16) + 1, SHAPE, ("select",)),
])
def test_cache_fields(L, field, value, expect, ops):
    run = calls(L, a_cache(**{field: value}), tokens())
    for op in ops:
        assert run[op]() == expect, op


@pytest.mark.parametrize("field,value,expect,ops", [
    ("cu_seqlens", None, NULL, ("attend", "append", "weigh")), ("q", None, NULL, ("attend", "weigh")),
    ("k", None, NULL, ("attend", "append")), ("v", None, NULL, ("attend", "append")),
    ("struct_size", 8, CACHE, ("attend", "append", "weigh")), ("total", 0, SHAPE, ("attend", "append", "weigh")),
    ("max_seqlen", 0, SHAPE, ("attend", "weigh")), ("max_seqlen", 129, SHAPE, ("attend",)),
    ("H", 0, SHAPE, ("attend", "weigh")), ("H", 5, CACHE, ("attend", "weigh")), ("H", 258, CACHE, ("attend", "weigh")),
    ("q", A + 8, ALIGN, ("attend", "weigh")), ("k", A + 4, ALIGN, ("attend", "append")),
    ("v", A + 4, ALIGN, ("attend", "append")), ("cu_seqlens", A + 2, ALIGN, ("attend", "append", "weigh")),
    ("q_strides", (256, 60), CACHE, ("attend", "weigh")), ("k_strides", (0, 64), CACHE, ("attend", "append")),
    ("v_strides", (128, -64), CACHE, ("attend", "append")),
])
def test_token_fields(L, field, value, expect, ops):
    run = calls(L, a_cache(), tokens(**{field: value}))
    for op in ops:
        assert run[op]() == expect, op


@pytest.mark.parametrize("kw,expect,ops", [
    (dict(c=None), NULL, ALL), (dict(x=None), NULL, ("attend", "append", "weigh")),
    (dict(o=None), NULL, ("attend",)), (dict(lse=None), NULL, ("attend", "weigh")), (dict(out=None), NULL, ("weigh",)),
    (dict(kept=None), NULL, ("select", "compact")), (dict(seq_pos=None), NULL, ("select",)),
    (dict(scale=0.0), SCALE, ("attend", "weigh")), (dict(scale=float("nan")), SCALE, ("attend", "weigh")),
    (dict(scale=1e-40), SCALE, ("weigh",)),
    (dict(o=A + 8), ALIGN, ("attend",)), (dict(lse=A + 2), ALIGN, ("attend", "weigh")),
    (dict(parents=A + 1), ALIGN, ("attend",)), (dict(out=A + 8), ALIGN, ("weigh",)),
    (dict(kept=A + 2), ALIGN, ("select", "compact")), (dict(seq_pos=A + 2), ALIGN, ("append", "select")),
    (dict(rows=A + 2, n_rows=3), ALIGN, ("append",)), (dict(rows=A, n_rows=0), SHAPE, ("append",)),
    (dict(budget=0), SHAPE, ("select", "compact")), (dict(recent=-1), SHAPE, ("select",)),
    (dict(recent=9), SHAPE, ("select",)),
    (dict(ws=None), WORKSPACE, ("attend",)), (dict(ws=A + 16), WORKSPACE, ("attend",)),
    (dict(ws_bytes=1000), WORKSPACE, ("attend",)),
])
def test_other_arguments(L, kw, expect, ops):
    kw = dict(kw)
    run = calls(L, kw.pop("c", a_cache()), kw.pop("x", tokens()), **kw)
    for op in ops:
        assert run[op]() == expect, op


def test_sizes_near_the_top_of_32_bits_are_refused(L):
    """The kernels round them up in 32 bits; up to 2^30 that is fine."""
    top, most = 2 ** 31 - 1, 2 ** 30
    one = a_cache(num_kv_heads=1, n_seq=1)
    for budget in (most + 1, top):
        run = calls(L, one, tokens(), budget=budget)
        assert run["select"]() == SHAPE and run["compact"]() == SHAPE
    assert calls(L, one, tokens(), budget=most, kept=A + 2)["compact"]() == ALIGN  # (not refused for its size)
    assert calls(L, one, tokens(total=top))["append"]() == SHAPE
    assert calls(L, one, tokens(), rows=A, n_rows=top)["append"]() == SHAPE
    assert calls(L, one, tokens(total=top, H=1))["weigh"]() == SHAPE


@pytest.mark.parametrize("opts", [dict(rescale_threshold=4.0), dict(poly_exp2_mask=0x11), dict(test_flags=2)])
def test_options_that_do_not_apply(L, opts):
    run = calls(L, a_cache(), tokens(), opts=attn.make_options(**opts))
    assert run["attend"]() == OPTION and run["weigh"]() == OPTION


def test_good_arguments_reach_the_device(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    run = calls(L, a_cache(), tokens())
    assert {run[op]() for op in ALL} == {ARCH}


def test_workspace_size(L):
    """One part of `rows` rows for each of the 640 ends of the CTAs' ranges."""
    size = cache.workspace_size
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731

    def expect(rows, d):
        return up(2049 * 4) + up(640 * rows * 8) + 640 * rows * d * 4

    assert size(32, 8, 1, 128) == expect(4, 128)
    assert size(14, 2, 128, 64) == expect(18 * 7, 64)     # 18 tokens of 7 heads in 128 rows
    assert size(8, 8, 128, 64) == expect(128, 64)
    for bad in ((8, 3, 1, 64), (8, 8, 0, 64), (8, 8, 129, 64), (8, 8, 1, 96), (258, 2, 1, 64), (0, 1, 1, 64)):
        assert size(*bad) == 0


def test_limits_match_the_header():
    src = open(HEADER).read()
    assert int(re.search(r"#define ATTN_CACHE_MAX_NEW (\d+)", src).group(1)) == cache.MAX_NEW
    m = re.search(r"#define ATTN_CACHE_MAX_SELECT \((\d+) << (\d+)\)", src)
    assert int(m.group(1)) << int(m.group(2)) == cache.MAX_SELECT


def test_compiled_binding_leaves_what_it_does_not_know_to_python(L):
    b = cache._load()
    t = torch.zeros(2, 2)
    for name, n, required in (("attend", 14, 9), ("append", 11, 7), ("weigh", 10, 8), ("select", 8, 5),
                              ("compact", 6, 4)):
        f = getattr(b, name)
        for args in ([t] * n, [3] * n, [None] * n, [t] * required + [None] * (n - required)):
            assert f(*args) is None
        with pytest.raises(TypeError):
            f(*[t] * (n - 1))


def test_binding_refuses_cpu_tensors_and_overlapping_rows():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 2, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(4, 2, 16)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cache.attn_fwd_cache(x, x, x, k, k, t, n, cu, 1)
    with pytest.raises(ValueError):
        cache.cache_append(x, x, k, k, t, n, cu)
    with pytest.raises(ValueError):
        cache.cache_weights(x, torch.zeros(2, 1), k, t, n, cu, 1, w)
    with pytest.raises(ValueError):
        cache.cache_select(w, t, n, 4)
    with pytest.raises(ValueError):
        cache.cache_compact(torch.zeros(1, 2, 4, dtype=torch.int32), k, k, t)
    with pytest.raises(ValueError):
        cache._strides(torch.zeros(1, 1, 64).expand(4, 3, 64))
    assert cache._strides(k) == (0, 0, 0)
    assert cache._strides(k.permute(0, 2, 1, 3)) == (2048, 64, 128)
    assert cache._strides(torch.zeros(5, 3, 64)[:, :1]) == (192, 64)
