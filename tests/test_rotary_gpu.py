"""Rotary positions on the GPU against their float64 definition and against differences."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_cache_reference as ref8
from cache_reference import HALF_BF16, f64
from exact_attention_63_gb300 import attn, rotary
from gpu_common import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need():
    need_gpu()


def close(got, x, positions, inv_freq, interleaved, magnitude, inverse=False):
    x = f64(x)
    want = ref8.rotary(x, positions, inv_freq, interleaved, magnitude, inverse)
    part = 2 * len(inv_freq)
    # One rounding to bf16, and of each pair's two elements: an angle of at most pi rounded to fp32 and
    # sines to 2 units (2^-22 together), two products and a sum in fp32 (3 x 2^-24); 2^-133 below bf16's range.
    other = np.zeros_like(x)
    u, w = (slice(0, part, 2), slice(1, part, 2)) if interleaved else (slice(0, part // 2), slice(part // 2, part))
    other[..., u] = other[..., w] = np.abs(x[..., u]) + np.abs(x[..., w])
    tol = HALF_BF16 * np.abs(want) + 2.0 ** -21 * other * abs(magnitude) * (1 + HALF_BF16) + 2.0 ** -133
    tol[..., part:] = 0
    assert (np.abs(f64(got) - want) <= tol).all(), (np.abs(f64(got) - want) - tol).max()


CASES = [  # batch, rows, H, H_kv, part of d, farthest position
    (1, 1, 8, 2, 1.0, 5), (2, 7, 4, 4, 0.5, 1000), (1, 64, 32, 8, 1.0, 131072), (3, 33, 1, 1, 0.25, 1 << 20),
    (1, 2500, 2, 1, 1.0, (1 << 31) - 1), (2, 1500, 3, 1, 0.5, 0),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotary(case, d, interleaved):
    batch, rows, H, hkv, share, far = case
    g = torch.Generator().manual_seed(rows)
    q, k = (torch.randn((batch, rows, h, d), generator=g).bfloat16().cuda() for h in (H, hkv))
    freq = rotary.rotary_frequencies(int(d * share), scaling="by_parts", factor=8.0)
    m = rotary.rotary_magnitude(8.0)
    positions = None
    if far:
        positions = torch.randint(-far - 1, far + 1, (batch, rows), generator=g).to(torch.int32)
        positions[0, 0] = far
    at = np.arange(rows)[None].repeat(batch, 0) if positions is None else positions.numpy()
    dev = None if positions is None else positions.cuda()
    for inverse, op in ((False, rotary.rotary_fwd), (True, rotary.rotary_bwd)):
        q2, k2 = op(q, k, dev, freq.cuda(), interleaved=interleaved, magnitude=m)
        close(q2, q, at, freq.tolist(), interleaved, m, inverse)
        close(k2, k, at, freq.tolist(), interleaved, m, inverse)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("part", [2, 4, 6, 8, 10, 12, 14, 16, 20, 24, 32, 40, 62, 64])
def test_every_access_width(part, d, interleaved):
    g = torch.Generator().manual_seed(part)
    q = torch.randn((1, 19, 3, d), generator=g).bfloat16().cuda()
    freq = rotary.rotary_frequencies(part).cuda()
    got, none = rotary.rotary_fwd(q, None, None, freq, interleaved=interleaved)
    assert none is None
    close(got, q, np.arange(19)[None], freq.tolist(), interleaved, 1.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_views_packed_rows_in_place_streams_and_graphs(interleaved):
    """Slices of a packed projection, [rows, heads, d] tensors, results over the inputs, another stream and a
    replayed graph all give the same bits."""
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn((2, 50, 12, 64), generator=g).bfloat16().cuda()
    q, k = qkv[:, :, :8], qkv[:, :, 8:10]
    pos = torch.randint(0, 9999, (2, 50), generator=g).to(torch.int32).cuda()
    freq = rotary.rotary_frequencies(32).cuda()
    kw = dict(interleaved=interleaved, magnitude=1.25)
    want = rotary.rotary_fwd(q.contiguous(), k.contiguous(), pos, freq, **kw)
    close(want[0], q, pos.cpu().numpy(), freq.tolist(), interleaved, 1.25)
    for got in (rotary.rotary_fwd(q, k, pos, freq, **kw), rotary.rotary_fwd(q, k, pos, freq, 1 if interleaved else 0, 1.25),
                rotary.rotary_fwd(qkv.flatten(0, 1)[:, :8], qkv.flatten(0, 1)[:, 8:10], pos.flatten(), freq, **kw)):
        assert torch.equal(got[0].view_as(want[0]), want[0]) and torch.equal(got[1].view_as(want[1]), want[1])
    rows = pos[0].contiguous()
    one = rotary.rotary_fwd(q, k, rows, freq, **kw)  # the same positions for both batches
    both = rotary.rotary_fwd(q, k, rows[None].repeat(2, 1), freq, **kw)
    assert torch.equal(one[0], both[0]) and torch.equal(one[1], both[1])
    for shape in ((), (0,)):  # strided views of one batch, of packed rows
        x = q[:1] if shape == () else q[0]
        y, _ = rotary.rotary_fwd(x, None, rows, freq, **kw)
        assert torch.equal(y.view_as(one[0][:1]), one[0][:1])
        z = torch.empty_like(qkv)[:1, :, :8] if shape == () else torch.empty_like(qkv)[0, :, :8]
        y, _ = rotary.rotary_fwd(x, None, rows, freq, q_out=z, **kw)
        assert y.data_ptr() == z.data_ptr() and torch.equal(y.reshape(one[0][:1].shape), one[0][:1])
    copy = qkv.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rotary.rotary_fwd(copy[:, :, :8], copy[:, :, 8:10], pos, freq, q_out=copy[:, :, :8], k_out=copy[:, :, 8:10], stream=side, **kw)
    side.synchronize()
    assert torch.equal(copy[:, :, :8], want[0]) and torch.equal(copy[:, :, 8:10], want[1])
    assert torch.equal(copy[:, :, 10:], qkv[:, :, 10:])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rotary.rotary_fwd(q, k, pos, freq, **kw)
    pos += 17
    graph.replay()
    want = rotary.rotary_fwd(q, k, pos, freq, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_far_positions_keep_their_angles():
    """Position p and frequency 2 pi / 2^20 at p and p + 2^20: the same turn, whatever p is."""
    q = torch.randn((1, 3, 1, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    freq = torch.full((32,), 2 * np.pi / 2 ** 20, dtype=torch.float64, device="cuda")
    near = torch.tensor([[5, 1000, 700001]], dtype=torch.int32, device="cuda")
    a, _ = rotary.rotary_fwd(q, None, near, freq)
    b, _ = rotary.rotary_fwd(q, None, near + (1 << 30), freq)
    # 2^30 times 2^-53 of a turn's 2^-20 is nothing; the tolerance is one rounding of each
    assert (f64(a) == f64(b)).mean() > 0.99 and np.abs(f64(a) - f64(b)).max() <= 2 * HALF_BF16 * np.abs(f64(a)).max()


def test_special_values_stay_in_their_pairs():
    q = torch.ones((1, 4, 2, 64)).bfloat16().cuda()
    q[0, 1, 0, 3], q[0, 2, 1, 40] = float("nan"), float("inf")
    freq = rotary.rotary_frequencies(32).cuda()
    y, _ = rotary.rotary_fwd(q, None, None, freq)
    bad = ~torch.isfinite(y)
    assert bad[0, 1, 0, [3, 19]].all() and bad[0, 2, 1, 40] and bad.sum() == 3


def test_gradients():
    """Those of q and k against the formula, and against differences of the float64 definition; a loss through
    rotary and attention trains."""
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((1, 40, h, 64), generator=g).bfloat16().cuda().requires_grad_() for h in (4, 2, 2))
    pos = torch.arange(100, 140, dtype=torch.int32).cuda()
    freq = rotary.rotary_frequencies(64).cuda()
    q2, k2 = rotary.rotary(q, k, pos, freq, magnitude=1.5)
    wq, wk = (torch.randn(x.shape, generator=g).bfloat16().cuda() for x in (q, k))
    ((q2 * wq).sum() + (k2 * wk).sum()).backward()
    at = pos.cpu().numpy()[None]
    close(q.grad, wq, at, freq.tolist(), False, 1.5, inverse=True)
    close(k.grad, wk, at, freq.tolist(), False, 1.5, inverse=True)
    x, w, step = f64(q), f64(wq), 2.0 ** -6
    for i in ((0, 3, 1, 5), (0, 39, 0, 40)):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        turned = [(ref8.rotary(y, at, freq.tolist(), False, 1.5) * w).sum() for y in (a, b)]
        # linear in x: the quotient is exact but for float64's rounding
        want = (turned[0] - turned[1]) / (2 * step)
        assert abs(float(q.grad[i]) - want) <= HALF_BF16 * abs(want) + 2.0 ** -20 * 1.5 * np.abs(w).max() * 2
    q.grad = k.grad = None
    q2, k2 = rotary.rotary(q, k, pos, freq)
    o, _ = attn.attention(q2, k2, v, causal=True)
    o.float().square().sum().backward()
    assert all(torch.isfinite(x.grad).all() and x.grad.abs().max() > 0 for x in (q, k, v))
    only, none = rotary.rotary(q, None, pos, freq)
    assert none is None
    only.sum().backward()


def test_backward_in_a_graph():
    g = torch.Generator().manual_seed(6)
    dq, dk = (torch.randn((2, 9, h, 128), generator=g).bfloat16().cuda() for h in (4, 2))
    freq = rotary.rotary_frequencies(128).cuda()
    want = rotary.rotary_bwd(dq, dk, None, freq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rotary.rotary_bwd(dq, dk, None, freq)
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals():
    freq = rotary.rotary_frequencies(64).cuda()
    q, k = torch.zeros((2, 5, 4, 64)).bfloat16().cuda(), torch.zeros((2, 5, 2, 64)).bfloat16().cuda()
    pos = torch.zeros(5, dtype=torch.int32).cuda()
    ok = lambda **kw: rotary.rotary_fwd(**{**dict(q=q, k=k, positions=pos, inv_freq=freq), **kw})  # noqa: E731
    ok()
    for kw in (dict(q=q.float()), dict(q=q.cpu()), dict(q=None), dict(k=k[:, :3]), dict(k=k.flatten(0, 1)), dict(positions=pos.long()),
               dict(positions=pos[:3]), dict(positions=torch.zeros((5, 2), dtype=torch.int32).cuda()), dict(inv_freq=freq.float()),
               dict(inv_freq=freq[None]), dict(q_out=torch.empty_like(k)), dict(k=None, k_out=k), dict(q=q.transpose(2, 3)),
               dict(q=q.expand(3, 2, 5, 4, 64)), dict(q=q[:1].expand(2, 5, 4, 64))):
        with pytest.raises(ValueError):
            ok(**kw)
    for kw in (dict(inv_freq=torch.zeros(33, dtype=torch.float64).cuda()), dict(magnitude=float("nan")), dict(magnitude=float("inf")),
               dict(q=torch.zeros((2, 5, 4, 32)).bfloat16().cuda(), k=None),
               dict(q=torch.zeros((2, 5, 4 * 64 + 4)).bfloat16().cuda()[..., :256].unflatten(2, (4, 64)), k=None)):
        with pytest.raises(attn.AttnError):
            ok(**kw)
    empty = ok(q=q[:, :0], k=k[:, :0], positions=pos[:0])
    assert empty[0].shape == (2, 0, 4, 64) and empty[1].shape == (2, 0, 2, 64)
