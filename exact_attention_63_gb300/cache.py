"""A key/value cache in pages and the operators on it: the binding of
``attn_fwd_cache`` and the ``attn_cache_*`` calls in ``include/attn_gb300.h``.

The tensors of a cache, all owned by the caller:

  k_cache, v_cache  bf16 [n_pages, page_size, H_kv, d], d = 64 or 128, page_size a
                    multiple of 16; strided views whose d is contiguous are fine
                    (pages stored [n_pages, H_kv, page_size, d], for instance)
  block_table       int32 [n_seq, max_blocks]: slot j of sequence s is slot
                    j % page_size of page block_table[s, j // page_size]
  seq_lens          int32 [n_seq]: sequence s holds slots [0, seq_lens[s])
  weights           fp32 [n_pages, H_kv, page_size]: attention weight gathered
  positions         int32 [n_pages, H_kv, page_size]: position of each slot's token
  seq_pos           int32 [n_seq]: tokens a sequence has ever appended

New tokens are packed: sequence s owns rows [cu_seqlens[s], cu_seqlens[s + 1]) of
q [total, H, d], k_new and v_new [total, H_kv, d].

A decoding step reads, in this order::

    o, lse = attn_fwd_cache(q, k_new, v_new, k_cache, v_cache, block_table, seq_lens, cu, max_new, parents)
    # ... the accepted rows of each sequence, packed by cu_acc ...
    seq_lens += n_accepted; seq_pos += n_accepted
    cache_append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, cu_acc, rows=accepted, ...)
    cache_weights(q[accepted], lse[:, accepted].contiguous(), k_cache, block_table, seq_lens, cu_acc, max_new, weights)
    # now and then:
    kept = cache_evict(k_cache, v_cache, weights, block_table, seq_lens, budget, recent, positions, seq_pos)
    seq_lens.clamp_(max=budget)

Argument marshalling only; the work runs in the library's CUDA kernels.  Lengths
and tables stay on the device, so every call can be captured into a CUDA graph and
replayed with other contents.  ``stream`` (default: the current one) is the stream
the call runs on, and the one its outputs and workspace are allocated on.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import attn

MAX_NEW = 128          # ATTN_CACHE_MAX_NEW
MAX_SELECT = 1 << 20   # ATTN_CACHE_MAX_SELECT

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


class Cache(ctypes.Structure):
    """Mirror of ``attn_cache``."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_strides", ctypes.c_longlong * 3), ("v_strides", ctypes.c_longlong * 3),
                ("weights", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_blocks", ctypes.c_int), ("n_seq", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("d", ctypes.c_int)]


class NewTokens(ctypes.Structure):
    """Mirror of ``attn_new_tokens``."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("q_strides", ctypes.c_longlong * 2), ("k_strides", ctypes.c_longlong * 2),
                ("v_strides", ctypes.c_longlong * 2), ("cu_seqlens", ctypes.c_void_p), ("total", ctypes.c_int),
                ("max_seqlen", ctypes.c_int), ("H", ctypes.c_int)]


def _need(name, t, dtype, dims, device, contiguous=True):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != dims or not t.is_cuda:
        raise ValueError(f"{name} must be a {dims}-D {dtype} CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if contiguous:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")


def _pages(name, t, device):
    _need(name, t, _BF16, 4, device, contiguous=False)


def _strides(t):
    """Element strides of all but the last dimension, for the library.  A stride
    of a dimension of one entry means nothing: the dense one stands for it."""
    if t.is_contiguous():
        return (0,) * (t.dim() - 1)
    out, dense = [], t.shape[-1]
    for i in range(t.dim() - 2, -1, -1):
        if t.shape[i] > 1 and t.stride(i) < t.shape[-1]:
            raise ValueError(f"overlapping rows: strides {tuple(t.stride())} of shape {tuple(t.shape)}")
        out.append(t.stride(i) if t.shape[i] > 1 else max(dense, 8))
        dense = max(dense, out[-1] * t.shape[i])
    return tuple(reversed(out))


def _cache_struct(k, v, block_table, seq_lens, weights, positions, hkv, d, n_pages, page_size):
    c = Cache()
    c.struct_size = ctypes.sizeof(Cache)
    if k is not None:
        c.k = k.data_ptr()
        c.k_strides[:] = _strides(k)
    if v is not None:
        c.v = v.data_ptr()
        c.v_strides[:] = _strides(v)
    if weights is not None:
        c.weights = weights.data_ptr()
    if positions is not None:
        c.positions = positions.data_ptr()
    c.block_table = block_table.data_ptr()
    if seq_lens is not None:
        c.seq_lens = seq_lens.data_ptr()
    c.n_pages, c.page_size, c.num_kv_heads, c.d = n_pages, page_size, hkv, d
    c.n_seq, c.max_blocks = block_table.shape
    return c


def _check_cache(k, v, block_table, seq_lens, weights=None, positions=None):
    """Types, shapes and devices of a cache's tensors; (device, H_kv, d, n_pages, page_size)."""
    lead = k if k is not None else weights
    if not isinstance(lead, torch.Tensor) or not lead.is_cuda:
        raise ValueError("the cache must be CUDA tensors")
    dev = lead.device
    if k is not None:
        _pages("k_cache", k, dev)
        n_pages, page_size, hkv, d = k.shape
        if v is not None:
            _pages("v_cache", v, dev)
            if v.shape != k.shape:
                raise ValueError(f"v_cache {tuple(v.shape)} must be shaped like k_cache {tuple(k.shape)}")
    else:
        _need("weights", weights, _F32, 3, dev)
        n_pages, hkv, page_size = weights.shape
        d = 0
    _need("block_table", block_table, _I32, 2, dev)
    if seq_lens is not None:
        _need("seq_lens", seq_lens, _I32, 1, dev)
        if seq_lens.shape[0] != block_table.shape[0]:
            raise ValueError("seq_lens and block_table must have as many sequences")
    for name, t, dt in (("weights", weights, _F32), ("positions", positions, _I32)):
        if t is not None:
            _need(name, t, dt, 3, dev)
            if tuple(t.shape) != (n_pages, hkv, page_size):
                raise ValueError(f"{name} must be [n_pages, H_kv, page_size] = {(n_pages, hkv, page_size)}")
    return dev, hkv, d, n_pages, page_size


def _check_seq(name, t, n, dev):
    _need(name, t, _I32, 1, dev)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries")


def _new_kv(k_new, v_new, hkv, d, dev):
    _need("k_new", k_new, _BF16, 3, dev, contiguous=False)
    _need("v_new", v_new, _BF16, 3, dev, contiguous=False)
    if k_new.shape != v_new.shape or tuple(k_new.shape[1:]) != (hkv, d):
        raise ValueError(f"k_new {tuple(k_new.shape)} and v_new {tuple(v_new.shape)} must be [total, {hkv}, {d}]")


class _on:
    """The tensors' device as the current one and `stream` as its current stream."""

    def __init__(self, dev, stream):
        self.cm = torch.cuda.stream(stream) if stream is not None else None
        self.dev = dev if dev.index != torch.cuda.current_device() else None

    def __enter__(self):
        if self.dev is not None:
            self.guard = torch.cuda.device(self.dev)
            self.guard.__enter__()
        if self.cm is not None:
            self.cm.__enter__()
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def __exit__(self, *a):
        if self.cm is not None:
            self.cm.__exit__(*a)
        if self.dev is not None:
            self.guard.__exit__(*a)


def _stream_fits(stream, dev):
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {dev}")


def workspace_size(H: int, H_kv: int, max_seqlen_q: int, d: int) -> int:
    """Bytes of attn_fwd_cache's workspace (0: the sizes are not supported)."""
    return int(attn.lib().attn_fwd_cache_workspace_size(H, H_kv, max_seqlen_q, d))


def attn_fwd_cache(q, k_new, v_new, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q: int,
                   parents=None, scale: float | None = None, out=None, lse=None, workspace=None, stream=None,
                   options=None):
    """Attention of new tokens over a paged cache and over each other.

    Token t of a sequence sees its seq_lens[s] cached keys, itself and its
    ancestors among the new tokens: ``parents`` (int32 [total], counted within the
    sequence, -1 = the last cached token) gives a drafted tree, None a chain.
    At most 128 new tokens a sequence; one is the usual decoding step.  q, k_new and
    v_new may be slices of a packed projection.  Returns (o [total, H, d] bf16,
    lse [H, total] fp32); rows that belong to no sequence are not written.
    ``workspace``: a uint8 tensor of workspace_size(...) bytes, else allocated.
    """
    dev, hkv, d, n_pages, page_size = _check_cache(k_cache, v_cache, block_table, seq_lens)
    if v_cache is None or seq_lens is None:
        raise ValueError("v_cache and seq_lens are needed")
    _need("q", q, _BF16, 3, dev, contiguous=False)
    _new_kv(k_new, v_new, hkv, d, dev)
    total, H = q.shape[0], q.shape[1]
    if k_new.shape[0] != total or q.shape[2] != d or H % hkv != 0:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k_new {tuple(k_new.shape)}, cache heads {hkv}, d {d}")
    _check_seq("cu_seqlens_q", cu_seqlens_q, block_table.shape[0] + 1, dev)
    if parents is not None:
        _check_seq("parents", parents, total, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _stream_fits(stream, dev)
    max_seqlen_q = int(max_seqlen_q)
    L = attn.lib()
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((total, H, d), dtype=_BF16, device=dev)
        else:
            _need("out", out, _BF16, 3, dev)
            if tuple(out.shape) != (total, H, d):
                raise ValueError("out must be shaped like q")
        if lse is None:
            lse = torch.empty((H, total), dtype=_F32, device=dev)
        else:
            _need("lse", lse, _F32, 2, dev)
            if tuple(lse.shape) != (H, total):
                raise ValueError("lse must be [H, total]")
        if total == 0:
            return out, lse
        if workspace is None:
            workspace = torch.empty(L.attn_fwd_cache_workspace_size(H, hkv, max_seqlen_q, d), dtype=torch.uint8,
                                    device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
        if options is not None:
            options.struct_size = ctypes.sizeof(attn.Options)
        c = _cache_struct(k_cache, v_cache, block_table, seq_lens, None, None, hkv, d, n_pages, page_size)
        x = NewTokens(ctypes.sizeof(NewTokens), q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), _strides(q),
                      _strides(k_new), _strides(v_new), cu_seqlens_q.data_ptr(), total, max_seqlen_q, H)
        rc = L.attn_fwd_cache(ctypes.byref(c), ctypes.byref(x), None if parents is None else parents.data_ptr(),
                              float(scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(),
                              ctypes.byref(options) if options is not None else None, s)
    attn._check(rc)
    return out, lse


def cache_append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, cu_new, rows=None, weights=None,
                 positions=None, seq_pos=None, stream=None):
    """Put new tokens' keys and values into the cache, in place.

    ``seq_lens`` (and ``seq_pos``) are the lengths after the append: token i of a
    sequence's n goes to slot seq_lens[s] - n + i, gets weight 0 and position
    seq_pos[s] - n + i (seq_lens where seq_pos is None).  ``rows`` (int32) picks rows
    of k_new and v_new, cu_new then counts entries of it: the accepted path of a
    drafted tree.
    """
    dev, hkv, d, n_pages, page_size = _check_cache(k_cache, v_cache, block_table, seq_lens, weights, positions)
    if v_cache is None or seq_lens is None:
        raise ValueError("v_cache and seq_lens are needed")
    _new_kv(k_new, v_new, hkv, d, dev)
    n_seq = block_table.shape[0]
    _check_seq("cu_new", cu_new, n_seq + 1, dev)
    if rows is not None:
        _need("rows", rows, _I32, 1, dev)
    if seq_pos is not None:
        _check_seq("seq_pos", seq_pos, n_seq, dev)
    _stream_fits(stream, dev)
    if k_new.shape[0] == 0 or (rows is not None and rows.shape[0] == 0):
        return
    with _on(dev, stream) as s:
        c = _cache_struct(k_cache, v_cache, block_table, seq_lens, weights, positions, hkv, d, n_pages, page_size)
        x = NewTokens(ctypes.sizeof(NewTokens), None, k_new.data_ptr(), v_new.data_ptr(), (0, 0), _strides(k_new),
                      _strides(v_new), cu_new.data_ptr(), k_new.shape[0], 0, 0)
        rc = attn.lib().attn_cache_append(ctypes.byref(c), ctypes.byref(x), None if rows is None else rows.data_ptr(),
                                          0 if rows is None else rows.shape[0],
                                          None if seq_pos is None else seq_pos.data_ptr(), s)
    attn._check(rc)


def cache_weights(q, lse, k_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q: int, weights=None,
                  scale: float | None = None, out=None, stream=None):
    """Add the attention weight that each cached key received from packed queries.

    The n queries of a sequence belong to its newest n cached tokens: query i sees
    slots up to seq_lens[s] - n + i.  lse [H, total] is theirs, as attn_fwd_varlen
    and attn_fwd_cache return it.  Writes weights + sums to ``out`` (default: into
    ``weights``) at every slot in use, and returns it; weights None counts as zeros
    (out is then needed).  Any number of queries: a decoded token, the last window
    of a prompt or the whole of it.
    """
    dev, hkv, d, n_pages, page_size = _check_cache(k_cache, None, block_table, seq_lens, weights)
    if seq_lens is None:
        raise ValueError("seq_lens is needed")
    if out is None:
        out = weights
    if out is None:
        raise ValueError("one of weights and out is needed")
    _need("out", out, _F32, 3, dev)
    if tuple(out.shape) != (n_pages, hkv, page_size):
        raise ValueError(f"out must be [n_pages, H_kv, page_size] = {(n_pages, hkv, page_size)}")
    _need("q", q, _BF16, 3, dev, contiguous=False)
    total, H = q.shape[0], q.shape[1]
    if q.shape[2] != d or H % hkv != 0:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, cache heads {hkv}, d {d}")
    _need("lse", lse, _F32, 2, dev)
    if tuple(lse.shape) != (H, total):
        raise ValueError(f"lse must be [H, total] = {(H, total)}")
    _check_seq("cu_seqlens_q", cu_seqlens_q, block_table.shape[0] + 1, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _stream_fits(stream, dev)
    with _on(dev, stream) as s:
        if total == 0:
            raise ValueError("q has no rows")
        c = _cache_struct(k_cache, None, block_table, seq_lens, weights, None, hkv, d, n_pages, page_size)
        x = NewTokens(ctypes.sizeof(NewTokens), q.data_ptr(), None, None, _strides(q), (0, 0), (0, 0),
                      cu_seqlens_q.data_ptr(), total, int(max_seqlen_q), H)
        rc = attn.lib().attn_cache_weights(ctypes.byref(c), ctypes.byref(x), lse.data_ptr(), float(scale),
                                           out.data_ptr(), s)
    attn._check(rc)
    return out


def cache_select(weights, block_table, seq_lens, budget: int, recent: int = 0, positions=None, seq_pos=None,
                 kept=None, stream=None):
    """Which tokens of each sequence and head stay when they may keep ``budget``.

    The ``recent`` newest (position >= seq_pos - recent; by slot where positions is
    None) come first, all alike, then the heaviest; of equals the lower slot.  Returns kept, int32
    [n_seq, H_kv, budget]: the slot that the token at slot i afterwards has now, -1
    behind the last.  Tokens that stay below slot ``budget`` keep their slot; the
    others fill the slots that become free, both ascending.
    """
    dev, hkv, _, n_pages, page_size = _check_cache(None, None, block_table, seq_lens, weights, positions)
    if seq_lens is None:
        raise ValueError("seq_lens is needed")
    n_seq = block_table.shape[0]
    if seq_pos is not None:
        _check_seq("seq_pos", seq_pos, n_seq, dev)
    elif positions is not None:
        raise ValueError("positions need seq_pos")
    budget, recent = int(budget), int(recent)
    _stream_fits(stream, dev)
    with _on(dev, stream) as s:
        if kept is None:
            kept = torch.empty((n_seq, hkv, max(budget, 0)), dtype=_I32, device=dev)
        else:
            _need("kept", kept, _I32, 3, dev)
            if tuple(kept.shape) != (n_seq, hkv, budget):
                raise ValueError(f"kept must be [n_seq, H_kv, budget] = {(n_seq, hkv, budget)}")
        c = _cache_struct(None, None, block_table, seq_lens, weights, positions, hkv, 0, n_pages, page_size)
        # (an empty tensor has no address: let the library answer for the budget)
        rc = attn.lib().attn_cache_select(ctypes.byref(c), None if seq_pos is None else seq_pos.data_ptr(), budget,
                                          recent, kept.data_ptr() or 16, s)
    attn._check(rc)
    return kept


def cache_compact(kept, k_cache, v_cache, block_table, weights=None, positions=None, stream=None):
    """Move the tokens that cache_select kept, in place: for every kept[s, h, i] >=
    budget (= kept.shape[2]) the key, value, weight and position of that slot go to
    slot i.  Set seq_lens to min(seq_lens, budget) afterwards."""
    dev, hkv, d, n_pages, page_size = _check_cache(k_cache, v_cache, block_table, None, weights, positions)
    if v_cache is None:
        raise ValueError("v_cache is needed")
    _need("kept", kept, _I32, 3, dev)
    if kept.shape[0] != block_table.shape[0] or kept.shape[1] != hkv or kept.shape[2] < 1:
        raise ValueError(f"kept must be [n_seq, H_kv, budget], not {tuple(kept.shape)}")
    _stream_fits(stream, dev)
    with _on(dev, stream) as s:
        c = _cache_struct(k_cache, v_cache, block_table, None, weights, positions, hkv, d, n_pages, page_size)
        rc = attn.lib().attn_cache_compact(ctypes.byref(c), kept.data_ptr(), kept.shape[2], s)
    attn._check(rc)


def cache_evict(k_cache, v_cache, weights, block_table, seq_lens, budget: int, recent: int = 0, positions=None,
                seq_pos=None, stream=None):
    """cache_select, then cache_compact: shrink every sequence and head to at most
    ``budget`` tokens, in place; returns kept.  The caller then clamps seq_lens to
    ``budget``."""
    kept = cache_select(weights, block_table, seq_lens, budget, recent, positions, seq_pos, stream=stream)
    cache_compact(kept, k_cache, v_cache, block_table, weights, positions, stream=stream)
    return kept
