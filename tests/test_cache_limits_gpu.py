"""Calls at the edges of what the cache operators' contract allows, on the GPU."""

from __future__ import annotations

import pytest
import torch

from cache_reference import Case
from exact_attention_63_gb300 import attn, cache
from gpu_common import need_gpu
from test_cache_gpu import check_attention

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
