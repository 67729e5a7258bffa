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

Argument marshalling only; the work runs in the library's CUDA kernels.  Dense
tensors take the short way through ``csrc/cache_bind.cpp``; strides, options, another
stream or device, and every refusal are dealt with here.  Lengths
and tables stay on the device, so every call can be captured into a CUDA graph and
replayed with other contents.  ``stream`` (default: the current one) is the stream
the call runs on, and the one its outputs and workspace are allocated on.
"""

from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import math
import os
import struct

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


# The structs as bytes in native layout.
_CACHE = struct.Struct("@N2P6q4P6i")
_TOKENS = struct.Struct("@N3P6qP3i0P")  # (0P: padded to a pointer's alignment, as in C)
_CACHE_SIZE, _TOKENS_SIZE = _CACHE.size, _TOKENS.size
assert _CACHE_SIZE == ctypes.sizeof(Cache) and _TOKENS_SIZE == ctypes.sizeof(NewTokens)

_BIND_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_cache_bind.so")
_bind = None


def _load():
    """The compiled binding (raises if it is missing or was built for another PyTorch)."""
    global _bind
    if not os.path.exists(_BIND_PATH):
        raise RuntimeError(f"{_BIND_PATH} is missing: build it with `python -m exact_attention_63_gb300.build`")
    attn.lib()
    loader = importlib.machinery.ExtensionFileLoader("_cache_bind", _BIND_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_cache_bind", loader))
    loader.exec_module(module)
    if not torch.__version__.startswith(module.torch_version):
        raise RuntimeError(f"{_BIND_PATH} was built for PyTorch {module.torch_version}, not {torch.__version__}: build it "
                           "again with `python -m exact_attention_63_gb300.build`")
    _bind = module
    return module


def _first(name, t):
    """The compiled binding, for the first call: t has to be what needs it."""
    _device(name, t)
    return _load()


def _refuse(name, t, dtype, dev, contiguous):
    """The reason why _need or _rows refused t."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, not {type(t).__name__}")
    if t.dtype != dtype or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of {dtype}, not {t.dtype} on {t.device}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name} must be contiguous" if contiguous else f"{name} must have a contiguous last dimension")


def _need(name, t, dtype, dev):
    """Address of t, a contiguous tensor of the type on CUDA device dev."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, dtype, dev, True)


def _rows(name, t, dev):
    """Address of t, a bf16 tensor on CUDA device dev whose last dimension is
    contiguous, and the element strides of the others for the library: (0, …) for
    dense ones."""
    try:
        if t.dtype is _BF16 and t.get_device() == dev:
            if t.is_contiguous():
                return t.data_ptr(), _DENSE[t.dim()]
            if t.stride(-1) == 1:
                return t.data_ptr(), _strides(t)
    except AttributeError:
        pass
    _refuse(name, t, _BF16, dev, False)


_DENSE = tuple((0,) * max(0, n - 1) for n in range(65))


def _strides(t):
    """The stride of a dimension of one entry means nothing; the dense one stands for it."""
    if t.is_contiguous():
        return _DENSE[t.dim()]
    shape, stride, out, dense = t.shape, t.stride(), [], t.shape[-1]
    for i in range(t.dim() - 2, -1, -1):
        if shape[i] > 1 and stride[i] < shape[-1]:
            raise ValueError(f"overlapping rows: strides {tuple(stride)} of shape {tuple(shape)}")
        out.append(stride[i] if shape[i] > 1 else max(dense, 8))
        dense = max(dense, out[-1] * shape[i])
    return tuple(reversed(out))


def _shape(name, t, n):
    """t's n sizes."""
    if not isinstance(t, torch.Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a {n}-D tensor")
    return t.shape


def _seq(name, t, n, dev):
    ptr = _need(name, t, _I32, dev)
    if t.shape != (n,):
        raise ValueError(f"{name} must have {n} entries, not shape {tuple(t.shape)}")
    return ptr


def _per_slot(name, t, dtype, shape, dev):
    ptr = _need(name, t, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be [n_pages, H_kv, page_size] = {tuple(shape)}, not {tuple(t.shape)}")
    return ptr


def _device(name, t):
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _pack_cache(dev, k, v, block_table, seq_lens, weights, positions):
    """attn_cache of the tensors, checked; (bytes, H_kv, d, n_seq).  What an operator
    does not use is None (k or weights is there)."""
    table = _need("block_table", block_table, _I32, dev)
    n_seq, max_blocks = _shape("block_table", block_table, 2)
    vp = wp = pp = lp = 0
    vs = (0, 0, 0)
    if k is not None:
        kp, ks = _rows("k_cache", k, dev)
        n_pages, page_size, hkv, d = _shape("k_cache", k, 4)
        if v is not None:
            vp, vs = _rows("v_cache", v, dev)
            if v.shape != k.shape:
                raise ValueError(f"v_cache {tuple(v.shape)} must be shaped like k_cache {tuple(k.shape)}")
    else:
        kp, ks, d = 0, vs, 0
        n_pages, hkv, page_size = _shape("weights", weights, 3)
    if weights is not None:
        wp = _per_slot("weights", weights, _F32, (n_pages, hkv, page_size), dev)
    if positions is not None:
        pp = _per_slot("positions", positions, _I32, (n_pages, hkv, page_size), dev)
    if seq_lens is not None:
        lp = _seq("seq_lens", seq_lens, n_seq, dev)
    return (_CACHE.pack(_CACHE_SIZE, kp, vp, *ks, *vs, wp, pp, table, lp, n_pages, page_size, max_blocks, n_seq, hkv,
                        d), hkv, d, n_seq)


def _pack_tokens(dev, q, k, v, cu, n_seq, hkv, d, max_seqlen):
    """attn_new_tokens of the tensors, checked; (bytes, total, H).  q, or k and v, may
    be None."""
    cp = _seq("cu_seqlens", cu, n_seq + 1, dev)
    qp = kp = vp = 0
    qs = ks = vs = (0, 0)
    total, H = None, hkv
    if q is not None:
        qp, qs = _rows("q", q, dev)
        total, H, dq = _shape("q", q, 3)
        if dq != d or not hkv or H % hkv != 0:
            raise ValueError(f"q {tuple(q.shape)} must be [total, H, {d}], H a multiple of {hkv}")
    if k is not None or v is not None:
        kp, ks = _rows("k_new", k, dev)
        vp, vs = _rows("v_new", v, dev)
        if total is None:
            total = _shape("k_new", k, 3)[0]
        if k.shape != (total, hkv, d) or v.shape != k.shape:
            raise ValueError(f"k_new {tuple(k.shape)} and v_new {tuple(v.shape)} must be [{total}, {hkv}, {d}]")
    return (_TOKENS.pack(_TOKENS_SIZE, qp, kp, vp, *qs, *ks, *vs, cp, total, max_seqlen, H), total, H)


def _elsewhere(dev, stream):
    """Whether a call has to switch device or stream first."""
    if stream is None:
        return torch._C._cuda_getDevice() != dev
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{dev}")
    return True


@contextlib.contextmanager
def _switched(dev, stream):
    """The tensors' device is current, and so is the stream: what is allocated inside
    belongs to it."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _options(options):
    if options is None:
        return None
    options.struct_size = ctypes.sizeof(attn.Options)
    return ctypes.byref(options)


def _stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


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
    ``options`` (attn.make_options): timeout_ms and the test flag apply.
    ``workspace``: a uint8 tensor of workspace_size(...) bytes, else allocated.
    """
    if stream is None and options is None:
        bind = _bind or _first("k_cache", k_cache)
        done = bind.attend(q, k_new, v_new, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q,
                           parents, scale, out, lse, workspace)
        if done.__class__ is tuple:
            return done
        if done is not None:
            attn._check(done)
    dev = _device("k_cache", k_cache)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return attn_fwd_cache(q, k_new, v_new, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q,
                                  max_seqlen_q, parents, scale, out, lse, workspace, None, options)
    if v_cache is None or seq_lens is None:
        raise ValueError("v_cache and seq_lens are needed")
    c, hkv, d, n_seq = _pack_cache(dev, k_cache, v_cache, block_table, seq_lens, None, None)
    if q is None or k_new is None or v_new is None:
        raise ValueError("q, k_new and v_new are needed")
    max_seqlen_q = int(max_seqlen_q)
    x, total, H = _pack_tokens(dev, q, k_new, v_new, cu_seqlens_q, n_seq, hkv, d, max_seqlen_q)
    par = None if parents is None else _seq("parents", parents, total, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is not None:
        _need("out", out, _BF16, dev)
        if out.shape != q.shape:
            raise ValueError("out must be shaped like q")
    if lse is not None:
        _need("lse", lse, _F32, dev)
        if lse.shape != (H, total):
            raise ValueError("lse must be [H, total]")
    if workspace is not None and (not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or
                                  not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    device = k_cache.device
    if out is None:
        out = torch.empty((total, H, d), dtype=_BF16, device=device)
    if lse is None:
        lse = torch.empty((H, total), dtype=_F32, device=device)
    if total == 0:
        return out, lse
    if workspace is None:
        workspace = torch.empty(workspace_size(H, hkv, max_seqlen_q, d), dtype=torch.uint8, device=device)
    rc = attn.lib().attn_fwd_cache(c, x, par, scale, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(),
                                   _options(options), _stream(dev))
    if rc:
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
    if stream is None:
        bind = _bind or _first("k_cache", k_cache)
        rc = bind.append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, cu_new, rows, weights, positions, seq_pos)
        if rc is not None:
            return attn._check(rc)
    dev = _device("k_cache", k_cache)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return cache_append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, cu_new, rows, weights, positions,
                                seq_pos)
    if v_cache is None or seq_lens is None:
        raise ValueError("v_cache and seq_lens are needed")
    c, hkv, d, n_seq = _pack_cache(dev, k_cache, v_cache, block_table, seq_lens, weights, positions)
    if k_new is None or v_new is None:
        raise ValueError("k_new and v_new are needed")
    x, total, _ = _pack_tokens(dev, None, k_new, v_new, cu_new, n_seq, hkv, d, 0)
    n_rows, rp = 0, None
    if rows is not None:
        rp = _need("rows", rows, _I32, dev)
        (n_rows,) = _shape("rows", rows, 1)
    sp = None if seq_pos is None else _seq("seq_pos", seq_pos, n_seq, dev)
    if total == 0 or (rows is not None and n_rows == 0):
        return
    rc = attn.lib().attn_cache_append(c, x, rp, n_rows, sp, _stream(dev))
    if rc:
        attn._check(rc)


def cache_weights(q, lse, k_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q: int, weights=None,
                  scale: float | None = None, out=None, stream=None, options=None):
    """Add the attention weight that each cached key received from packed queries.

    The n queries of a sequence belong to its newest n cached tokens: query i sees
    slots up to seq_lens[s] - n + i.  lse [H, total] is theirs, as attn_fwd_varlen
    and attn_fwd_cache return it.  Writes weights + sums to ``out`` (default: into
    ``weights``) at every slot in use, and returns it; weights None counts as zeros
    (out is then needed).  Any number of queries: a decoded token, the last window
    of a prompt or the whole of it; none at all adds nothing.  ``scale`` is at least
    1e-30.
    """
    if stream is None and options is None:
        into = weights if out is None else out
        bind = _bind or _first("k_cache", k_cache)
        rc = bind.weigh(q, lse, k_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q, into, weights, scale)
        if rc is not None:
            attn._check(rc)
            return into
    dev = _device("k_cache", k_cache)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return cache_weights(q, lse, k_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q, weights, scale, out, None,
                                 options)
    if seq_lens is None:
        raise ValueError("seq_lens is needed")
    c, hkv, d, n_seq = _pack_cache(dev, k_cache, None, block_table, seq_lens, weights, None)
    if out is None:
        out = weights
    if out is None:
        raise ValueError("one of weights and out is needed")
    op = _per_slot("out", out, _F32, (k_cache.shape[0], hkv, k_cache.shape[1]), dev)
    if q is None:
        raise ValueError("q is needed")
    x, total, H = _pack_tokens(dev, q, None, None, cu_seqlens_q, n_seq, hkv, d, int(max_seqlen_q))
    lp = _need("lse", lse, _F32, dev)
    if lse.shape != (H, total):
        raise ValueError(f"lse must be [H, total] = {(H, total)}")
    if total == 0:  # what there was at every slot in use
        if weights is not None and op == weights.data_ptr():
            return out
        # (the library takes no empty tensors: a row that adds nothing stands for them)
        q, lse = q.new_zeros((1, H, d)), lse.new_full((H, 1), math.inf)
        x, lp = _pack_tokens(dev, q, None, None, cu_seqlens_q, n_seq, hkv, d, 1)[0], lse.data_ptr()
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    rc = attn.lib().attn_cache_weights(c, x, lp, scale, op, _options(options), _stream(dev))
    if rc:
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
    if stream is None:
        bind = _bind or _first("weights", weights)
        done = bind.select(weights, block_table, seq_lens, budget, recent, positions, seq_pos, kept)
        if done.__class__ is int:
            attn._check(done)
        elif done is not None:
            return done
    dev = _device("weights", weights)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return cache_select(weights, block_table, seq_lens, budget, recent, positions, seq_pos, kept)
    if seq_lens is None:
        raise ValueError("seq_lens is needed")
    c, hkv, _, n_seq = _pack_cache(dev, None, None, block_table, seq_lens, weights, positions)
    if positions is not None and seq_pos is None:
        raise ValueError("positions need seq_pos")
    sp = None if seq_pos is None else _seq("seq_pos", seq_pos, n_seq, dev)
    budget, recent = int(budget), int(recent)
    if kept is not None:
        _need("kept", kept, _I32, dev)
        if kept.shape != (n_seq, hkv, budget):
            raise ValueError(f"kept must be [n_seq, H_kv, budget] = {(n_seq, hkv, budget)}")
    if kept is None:
        kept = torch.empty((n_seq, hkv, max(budget, 0)), dtype=_I32, device=weights.device)
    # (an empty tensor has no address: the library answers for the budget)
    rc = attn.lib().attn_cache_select(c, sp, budget, recent, kept.data_ptr() or 16, _stream(dev))
    if rc:
        attn._check(rc)
    return kept


def cache_compact(kept, k_cache, v_cache, block_table, weights=None, positions=None, stream=None):
    """Move the tokens that cache_select kept, in place: for every kept[s, h, i] >=
    budget (= kept.shape[2]) the key, value, weight and position of that slot go to
    slot i.  Set seq_lens to min(seq_lens, budget) afterwards."""
    if stream is None:
        bind = _bind or _first("k_cache", k_cache)
        rc = bind.compact(kept, k_cache, v_cache, block_table, weights, positions)
        if rc is not None:
            return attn._check(rc)
    dev = _device("k_cache", k_cache)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return cache_compact(kept, k_cache, v_cache, block_table, weights, positions)
    if v_cache is None:
        raise ValueError("v_cache is needed")
    c, hkv, _, n_seq = _pack_cache(dev, k_cache, v_cache, block_table, None, weights, positions)
    kp = _need("kept", kept, _I32, dev)
    if kept.dim() != 3 or kept.shape[:2] != (n_seq, hkv) or kept.shape[2] < 1:
        raise ValueError(f"kept must be [n_seq, H_kv, budget], not {tuple(kept.shape)}")
    rc = attn.lib().attn_cache_compact(c, kp, kept.shape[2], _stream(dev))
    if rc:
        attn._check(rc)


def cache_evict(k_cache, v_cache, weights, block_table, seq_lens, budget: int, recent: int = 0, positions=None,
                seq_pos=None, stream=None):
    """cache_select, then cache_compact: shrink every sequence and head to at most
    ``budget`` tokens, in place; returns kept.  The caller then clamps seq_lens to
    ``budget``."""
    kept = cache_select(weights, block_table, seq_lens, budget, recent, positions, seq_pos, stream=stream)
    cache_compact(kept, k_cache, v_cache, block_table, weights, positions, stream=stream)
    return kept
