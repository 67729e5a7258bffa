"""Calls at the edges of what the cache operators' contract allows, on the GPU."""

from __future__ import annotations

import pytest
import torch

from cache_reference import Case, f64
from exact_attention_63_gb300 import attn, cache
from gpu_common import need_gpu
from test_cache_gpu import check_attention, check_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    need_gpu()
    assert attn.get_status() == 0
    yield
    assert attn.get_status() == 0


@pytest.mark.parametrize("most", [8, 33, 40, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_fewer_tokens_than_max_seqlen(d, most):
    """max_seqlen is a bound: above total, and above every sequence's tokens."""
    c = Case([300, 40, 129], [3, 1, 4], 8, 2, d, 16, seed=50).cuda()
    args = (c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu)
    ws = torch.empty(cache.workspace_size(8, 2, 128, d), dtype=torch.uint8, device="cuda")  # for every max_seqlen
    for kw in (dict(), dict(workspace=ws), dict(stream=torch.cuda.current_stream())):
        o, lse = cache.attn_fwd_cache(*args, most, parents=c.parents, **kw)
        check_attention(c, o, lse)


def test_attention_of_one_full_row_tile_with_room_for_two():
    """30 rows of 4 heads under a bound of 40: total decides on one row tile a CTA, which leaves more
    parts than two would."""
    c = Case([700], [30], 8, 2, 128, 16, seed=51).cuda()
    for kw in (dict(), dict(stream=torch.cuda.current_stream())):
        o, lse = cache.attn_fwd_cache(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.seq_lens, c.cu, 40, parents=c.parents, **kw)
        check_attention(c, o, lse)


def test_wait_limit_where_a_loader_is_done():
    """One chunk of rows a tile: the rows' loader has issued all its copies when the waits for the
    withheld keys run out.  Each call ends, and the next one is right."""
    c = Case([200, 90, 256], [1, 2, 1], 8, 2, 128, 16, seed=52).cuda()
    start, lse = f64(c.weights), torch.full((8, c.total), 6.0, device="cuda")
    opts = attn.make_options(timeout_ms=1, test_flags=attn.TEST_WITHHOLD_KV)
    for _ in range(10):
        cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 2, c.weights, out=torch.zeros_like(c.weights), options=opts)
        assert attn.get_status() == -8
        out = cache.cache_weights(c.q, lse, c.k, c.table, c.seq_lens, c.cu, 2, c.weights, out=torch.zeros_like(c.weights))
        check_weights(c, lse, start, out)
