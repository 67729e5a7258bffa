"""attn.attention under create_graph, with the two kernels' places taken by plain CPU code."""

from __future__ import annotations

import pytest
import torch

from exact_attention_63_gb300 import attn


def forward(q, k, v, causal, scale, causal_align):
    assert not causal and scale is None and causal_align == "top-left"
    z = torch.einsum("bqhd,bkhd->bhqk", q, k) / q.shape[-1] ** 0.5
    return torch.einsum("bhqk,bkhd->bqhd", z.softmax(-1), v), z.logsumexp(-1)


def backward(q, k, v, o, lse, do, causal, scale, causal_align, deterministic):
    with torch.enable_grad():
        x = [t.detach().requires_grad_() for t in (q, k, v)]
        return torch.autograd.grad(forward(*x, causal, scale, causal_align)[0], x, do.detach())


@pytest.fixture
def plain(monkeypatch):
    monkeypatch.setattr(attn, "attn_fwd", forward)
    monkeypatch.setattr(attn, "attn_bwd", backward)
    g = torch.Generator().manual_seed(0)
    return [torch.randn((1, 5, 2, 8), generator=g, dtype=torch.float64).requires_grad_() for _ in range(3)]


def test_gradients_of_gradients_are_refused(plain):
    """attn_bwd has no gradient: a penalty on the first ones must not lose its term without a word, least of all
    where another way leads to the same leaves."""
    o, _ = attn.attention(*plain)
    first = torch.autograd.grad((o ** 2).sum() + (plain[0] ** 4).sum(), plain, create_graph=True)
    want = torch.autograd.grad((forward(*plain, False, None, "top-left")[0] ** 2).sum() + (plain[0] ** 4).sum(), plain)
    for a, b in zip(first, want):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (first[0] ** 2).sum().backward()


def test_first_gradients_are_as_they_were(plain):
    o, lse = attn.attention(*plain)
    assert not lse.requires_grad
    (o ** 2).sum().backward()
    want = torch.autograd.grad((forward(*plain, False, None, "top-left")[0] ** 2).sum(), plain)
    for x, b in zip(plain, want):
        assert torch.allclose(x.grad, b, rtol=1e-12, atol=1e-12) and not x.grad.requires_grad
