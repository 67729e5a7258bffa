"""Gradients of the rotary positions' gradients: on the CPU with the turn in plain float64 in the kernel's place,
and on the GPU."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_cache_reference as ref8
from cache_reference import HALF_BF16, f64
from exact_attention_63_gb300 import rotary
from gpu_common import need_gpu


def plain_turn(q, k, positions, inv_freq, interleaved, magnitude, q_out, k_out, inverse, stream):
    """rotary._turn in float64, and as little a part of any autograd graph as a kernel's launch."""
    assert q_out is None and k_out is None and stream is None
    at = np.arange(q.shape[1])[None].repeat(q.shape[0], 0) if positions is None else positions.numpy()
    one = lambda x: None if x is None else torch.from_numpy(  # noqa: E731
        ref8.rotary(x.detach().numpy(), at, inv_freq.tolist(), interleaved, magnitude, inverse))
    return one(q), one(k)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("with_k", [False, True])
def test_second_derivatives_by_differences(monkeypatch, interleaved, with_k):
    monkeypatch.setattr(rotary, "_turn", plain_turn)
    g = torch.Generator().manual_seed(1)
    q = torch.randn((2, 3, 2, 8), generator=g, dtype=torch.float64).requires_grad_()
    k = torch.randn((2, 3, 1, 8), generator=g, dtype=torch.float64).requires_grad_()
    pos, freq = torch.tensor([[0, 5, 1000], [7, 7, 2]]), rotary.rotary_frequencies(6)
    both = (q, k) if with_k else (q,)

    def turned(*x):
        y = rotary.rotary(x[0], x[1] if with_k else None, pos, freq, interleaved, 1.5)
        return tuple(t.sin() for t in y if t is not None)  # (so that second derivatives are not zero)

    assert torch.autograd.gradcheck(turned, both)
    assert torch.autograd.gradgradcheck(turned, both)


def test_a_penalty_on_gradients_keeps_its_term(monkeypatch):
    """With another way from the loss to the inputs, a lost term would show in nothing but the values."""
    monkeypatch.setattr(rotary, "_turn", plain_turn)
    g = torch.Generator().manual_seed(2)
    q = torch.randn((1, 4, 2, 8), generator=g, dtype=torch.float64).requires_grad_()
    freq = rotary.rotary_frequencies(8)

    def grads(turn):
        y = turn(q)
        (dq,) = torch.autograd.grad((y ** 3).sum() + (q ** 4).sum(), q, create_graph=True)
        return torch.autograd.grad((dq ** 2).sum(), q)[0]

    def formula(x):
        a = torch.arange(4, dtype=torch.float64)[:, None, None] * freq
        u, w = x[..., :4], x[..., 4:]
        return torch.cat([u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()], -1)

    got, want = grads(lambda x: rotary.rotary(x, None, None, freq)[0]), grads(formula)
    assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_second_derivatives_on_the_gpu(interleaved):
    """L = sum of y^3, y the turned q; the gradient of sum(c * dL/dq), c fixed, is the turn back of 6 y (c turned)."""
    need_gpu()
    g = torch.Generator().manual_seed(3)
    q, c = (torch.randn((2, 9, 3, 64), generator=g).bfloat16().cuda() for _ in range(2))
    q.requires_grad_()
    freq, m = rotary.rotary_frequencies(32).cuda(), 1.25
    y, _ = rotary.rotary(q, None, None, freq, interleaved, m)
    (dq,) = torch.autograd.grad((y.float() ** 3).sum(), q, create_graph=True)
    (dq.float() * c).sum().backward()
    at = np.arange(9)[None].repeat(2, 0)
    turn = lambda x, inverse=False: ref8.rotary(x, at, freq.tolist(), interleaved, m, inverse)  # noqa: E731
    # y, the turned c and their product are each rounded to bf16 once, before the last turn adds two of them.
    # The turns' own arithmetic is off by 2^-21 of a pair's two sizes (twice here, and in the last turn).
    pairs = lambda x: pair_sum(np.abs(x), 32, interleaved)  # noqa: E731
    Y, C = turn(f64(q)), turn(f64(c))
    off_y, off_c = (HALF_BF16 * np.abs(t) + 2.0 ** -21 * m * pairs(x) for t, x in ((Y, f64(q)), (C, f64(c))))
    P = 6 * Y * C
    off_p = 6 * (off_y * np.abs(C) + off_c * np.abs(Y) + off_y * off_c)
    off_p = off_p + (HALF_BF16 + 2.0 ** -22) * (np.abs(P) + off_p)
    want = turn(P, True)
    tol = m * pairs(off_p) + 2.0 ** -21 * m * pairs(np.abs(P) + off_p)
    tol[..., 32:] = off_p[..., 32:]
    tol = tol + HALF_BF16 * (np.abs(want) + tol)
    assert (np.abs(f64(q.grad) - want) <= tol).all()
    assert np.abs(want).max() > 4 * tol.max()  # (a lost term would not pass)


def pair_sum(x, part, interleaved):
    """In each place of a pair the sum of the pair's two; elements beyond `part` as they are."""
    y = x.copy()
    u, w = (slice(0, part, 2), slice(1, part, 2)) if interleaved else (slice(0, part // 2), slice(part // 2, part))
    y[..., u] = y[..., w] = x[..., u] + x[..., w]
    return y


@pytest.mark.gpu
def test_a_side_without_heads_leaves_the_other_as_it_is():
    """k (or q) of no heads has nothing to turn; q (or k) is turned all the same, forward and back."""
    need_gpu()
    g = torch.Generator().manual_seed(4)
    x = torch.randn((2, 9, 3, 64), generator=g).bfloat16().cuda()
    none = x[:, :, :0]
    freq = rotary.rotary_frequencies(64).cuda()
    for op in (rotary.rotary_fwd, rotary.rotary_bwd):
        want, _ = op(x, None, None, freq)
        for out in (None, torch.full_like(x, 7.0)):
            (a, b), (c, d) = op(x, none, None, freq, q_out=out), op(none, x, None, freq, k_out=out)
            assert torch.equal(a, want) and torch.equal(d, want) and b.shape == c.shape == none.shape
            assert out is None or (a is out and d is out)
    x.requires_grad_()
    y, _ = rotary.rotary(x, none, None, freq)
    y.sum().backward()
    assert torch.equal(x.grad, rotary.rotary_bwd(torch.ones_like(x), None, None, freq)[0])
