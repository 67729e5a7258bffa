"""Rotary positions on q and k: the binding of ``attn_rotary`` in ``include/attn_gb300.h``.

With the angle a = position * inv_freq[i], pair i of the first rotary_dim elements of every head
turns from (u, w) to m (u cos a - w sin a, w cos a + u sin a); the elements behind stay.  Pairs are
the neighbours (2i, 2i + 1) (``interleaved``) or (i, i + rotary_dim / 2).

``rotary_frequencies`` makes inv_freq for the usual ways of reaching longer contexts; any float64
tensor of radians a position will do.  ``rotary`` has gradients, ``rotary_fwd`` and ``rotary_bwd`` are
its two directions; results may be written over the inputs.  Angles of far positions lose
nothing: they are taken modulo a turn in 64 bits.

Calls go through ``csrc/cache_bind.cpp`` like those of ``cache.py``, so the compiled binding has to be
there (``attn.py`` alone does not need it).
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import attn, cache

_BF16, _I32 = torch.bfloat16, torch.int32


class Rows(ctypes.Structure):
    """Mirror of ``attn_rows``."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("x_strides", ctypes.c_longlong * 3), ("y_strides", ctypes.c_longlong * 3), ("heads", ctypes.c_int)]


SCALINGS = ("none", "linear", "base", "by_parts")


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_length: int = 4096, turns=(32.0, 1.0), device=None):
    """inv_freq, float64 [rotary_dim / 2]: base^(-2i / rotary_dim), stretched for contexts ``factor``
    times the ``original_length`` that a model was trained on.

    scaling "linear" divides all by factor; "base" raises the base so that the slowest pair is
    divided by factor and the fastest stays; "by_parts" divides the pairs that turn at most
    turns[1] times over the original length, leaves those that turn at least turns[0] times, and
    goes from one to the other linearly in i (usually with the magnitude of
    ``rotary_magnitude(factor)``): the interpolation of Peng, Quesnelle, Fan and Shippole, "YaRN:
    efficient context window extension of large language models", 2023.
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {SCALINGS}")
    if not (math.isfinite(base) and base > 1.0 and math.isfinite(factor) and factor > 0.0):
        raise ValueError("base must be above 1 and factor positive, both finite")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    if scaling == "base":
        if rotary_dim < 4:
            raise ValueError("scaling by the base needs two pairs at least")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        fast, slow = turns
        if not fast > slow > 0.0:
            raise ValueError("turns must be two positive numbers, the larger first")
        at = [rotary_dim * math.log(original_length / (t * 2.0 * math.pi)) / (2.0 * math.log(base)) for t in (fast, slow)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary_dim - 1)
        keep = 1.0 - torch.clamp((i - low) / max(high - low, 0.001), 0.0, 1.0)
        f = f / factor * (1.0 - keep) + f * keep
    return f.to(device) if device is not None else f


def rotary_magnitude(factor: float) -> float:
    """The usual magnitude of frequencies scaled by parts: 0.1 ln(factor) + 1, 1 up to a factor of 1."""
    return 1.0 if factor <= 1.0 else 0.1 * math.log(factor) + 1.0


def _side(name, t, dev):
    """The tensor's address and (batch, row, head) strides, batch and rows, heads, d."""
    if not isinstance(t, torch.Tensor) or t.dtype != _BF16 or t.get_device() != dev or t.dim() not in (3, 4) or \
            (t.numel() and t.stride(-1) != 1):
        raise ValueError(f"{name} must be a bf16 CUDA tensor (batch, seq, heads, head_dim) or (rows, heads, head_dim) "
                         f"on cuda:{dev} with a contiguous head_dim")
    shape = t.shape if t.dim() == 4 else (1, *t.shape)
    st = cache._strides(t) if t.numel() else (0,) * (t.dim() - 1)
    if t.dim() == 3 and any(st):
        st = (max(8, st[0] * t.shape[0]), *st)
    return t.data_ptr(), st if t.dim() == 4 or any(st) else (0, 0, 0), shape


def _turn(q, k, positions, inv_freq, interleaved, magnitude, q_out, k_out, inverse, stream):
    if stream is None:
        bind = cache._bind or cache._first("q", q)
        done = bind.rotary(q, k, positions, inv_freq, interleaved, magnitude, q_out, k_out, inverse)
        if done.__class__ is tuple:
            return done
        if done is not None:
            attn._check(done)
    dev = cache._device("q", q)
    if cache._elsewhere(dev, stream):
        with cache._switched(dev, stream):
            return _turn(q, k, positions, inv_freq, interleaved, magnitude, q_out, k_out, inverse, None)
    if k is None and k_out is not None:
        raise ValueError("k_out needs k")
    sides, outs = [], []
    for name, t, out in (("q", q, q_out), ("k", k, k_out)):
        if t is None:
            outs.append(None)
            continue
        ptr, st, shape = _side(name, t, dev)
        if out is None:
            out = torch.empty(t.shape, dtype=_BF16, device=t.device)
        optr, ost, oshape = _side(name + "_out", out, dev)
        if out.shape != t.shape:
            raise ValueError(f"{name}_out must be shaped like {name}")
        if sides and (t.dim() != q.dim() or shape[:2] != sides[0][2][:2] or shape[3] != sides[0][2][3]):
            raise ValueError(f"k {tuple(k.shape)} must be shaped like q {tuple(q.shape)} but for the heads")
        r = Rows()
        r.struct_size = ctypes.sizeof(Rows)
        r.x, r.y, r.heads = ptr, optr, shape[2]
        r.x_strides[:], r.y_strides[:] = st, ost
        sides.append((r, out, shape))
        outs.append(out)
    batch, rows, _, d = sides[0][2]
    fp = cache._need("inv_freq", inv_freq, torch.float64, dev)
    (pairs,) = cache._shape("inv_freq", inv_freq, 1)
    pp, ps = None, 0
    if positions is not None:
        pp = cache._need("positions", positions, _I32, dev)
        if positions.shape == (batch, rows) and q.dim() == 4:
            ps = rows
        elif positions.shape != (rows,):
            raise ValueError(f"positions must be [{rows}]" + (f" or [{batch}, {rows}]" if q.dim() == 4 else "") +
                             f", not {tuple(positions.shape)}")
    turned = [ctypes.byref(r) for r, _, shape in sides if shape[2]]
    if batch * rows == 0 or not turned:
        return tuple(outs)
    rc = attn.lib().attn_rotary(turned[0], turned[1] if len(turned) > 1 else None, batch, rows, d, pp, ps, fp, 2 * pairs,
                                int(bool(interleaved)), float(magnitude), int(inverse), cache._stream(dev))
    if rc:
        attn._check(rc)
    return tuple(outs)


def rotary_fwd(q, k, positions, inv_freq, interleaved: bool = False, magnitude: float = 1.0, q_out=None, k_out=None,
               stream=None):
    """Turn q and k (k may be None) by their positions; returns (q', k').

    q [batch, seq, H, d] and k [batch, seq, H_kv, d], or packed [rows, H, d] and [rows, H_kv, d], bf16,
    strided views such as slices of a packed projection allowed; ``positions`` int32 [seq] or
    [batch, seq] ([rows] where packed), None: the row's number; ``inv_freq`` float64
    [rotary_dim / 2].  The results are dense, or written to ``q_out`` and ``k_out``, which may be q
    and k themselves.
    """
    return _turn(q, k, positions, inv_freq, interleaved, magnitude, q_out, k_out, False, stream)


def rotary_bwd(dq, dk, positions, inv_freq, interleaved: bool = False, magnitude: float = 1.0, q_out=None, k_out=None,
               stream=None):
    """Gradients of q and k from those of rotary_fwd's results: the turn back, with the same factor."""
    return _turn(dq, dk, positions, inv_freq, interleaved, magnitude, q_out, k_out, True, stream)


class _Rotary(torch.autograd.Function):
    """The turn, or the turn back (``inverse``): each is the other's gradient."""

    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, interleaved, magnitude, inverse):
        ctx.save_for_backward(positions, inv_freq)
        ctx.cfg = (interleaved, magnitude, inverse)
        return _turn(q, k, positions, inv_freq, interleaved, magnitude, None, None, inverse, None)

    @staticmethod
    def backward(ctx, dq, dk):
        positions, inv_freq = ctx.saved_tensors
        interleaved, magnitude, inverse = ctx.cfg
        dq, dk = dq.contiguous(), None if dk is None else dk.contiguous()
        if torch.is_grad_enabled():  # (create_graph: the gradients have gradients)
            grads = _Rotary.apply(dq, dk, positions, inv_freq, interleaved, magnitude, not inverse)
        else:
            grads = _turn(dq, dk, positions, inv_freq, interleaved, magnitude, None, None, not inverse, None)
        return (*grads, None, None, None, None, None)


def rotary(q, k, positions, inv_freq, interleaved: bool = False, magnitude: float = 1.0):
    """rotary_fwd with gradients to q and k, of any order; what attn.attention then takes."""
    return _Rotary.apply(q, k, positions, inv_freq, interleaved, magnitude, False)
