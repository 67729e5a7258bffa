"""Page tables at the ends of their sizes, and captured with more tokens than the tables' own kernel places."""

from __future__ import annotations

import pytest
import torch

from exact_attention_63_gb300 import cache
from gpu_common import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need():
    need_gpu()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_tables_of_nearly_two_to_the_31_entries():
    """All pages go back and come again: their numbers, rounded up to the warps' runs, pass 2^31."""
    n, width, page = 33, 65075262, 16
    pages = n * width
    assert 2 ** 31 - 4096 < pages < 2 ** 31 and width * page <= 2 ** 30
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(n, width)
    free = torch.full((pages,), -7, dtype=torch.int32, device="cuda")
    held, top = ints(*[width] * n), ints(0)
    missing, _, _ = cache.cache_pages(ints(*[0] * n), table, held, free, top, page)
    assert top.item() == pages and held.tolist() == missing.tolist() == [0] * n
    assert bool((table == -1).all()) and bool((free == torch.arange(pages, dtype=torch.int32, device="cuda")).all())
    missing, _, _ = cache.cache_pages(ints(*[width * page] * n), table, held, free, top, page)
    assert top.item() == 0 and missing.tolist() == [0] * n and held.tolist() == [width] * n
    assert bool((table.flatten() == torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")).all())
    del table, free
    torch.cuda.empty_cache()


def test_prompts_in_a_graph():
    """The tables' cluster and the slots' kernel, captured and replayed with other lengths."""
    width, page = 600, 16
    table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    free, held, top = torch.arange(1500, dtype=torch.int32, device="cuda"), ints(0, 0, 0), ints(1500)
    lens, cu, total = ints(9000, 30, 7), ints(0, 9000, 9010, 9017), 9020
    out = ints(0, 0, 0), torch.full((total,), -9, dtype=torch.int64, device="cuda"), torch.full((total,), -9, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.cache_pages(lens, table, held, free, top, page, cu, total, *out)
    for want in ([9000, 30, 7], [17, 9600, 100], [9600, 9600, 5], [0, 0, 0]):
        lens.copy_(ints(*want))
        before = [t.clone() for t in (table, held, free, top)]
        graph.replay()
        got = [t.clone() for t in (*out, table, held, free, top)]
        for t, x in zip((table, held, free, top), before):
            t.copy_(x)
        eager = cache.cache_pages(lens, table, held, free, top, page, cu, total, *[t.clone() for t in out])
        for x, y in zip(got, (*eager, table, held, free, top)):
            assert torch.equal(x, y)
        blocks = [-(-a // page) for a in want]
        # (sequences in order as long as 1500 pages last)
        assert out[0].tolist() == [0 if sum(blocks[:s + 1]) <= 1500 else blocks[s] - int(held[s]) for s in range(3)]
        slot = torch.arange(9000) + want[0] - 9000
        assert torch.equal(out[2][:9000].cpu(), slot.int()) and out[1][9017:].tolist() == [-9] * 3
        live = slot >= 0
        at = table.cpu()[0, slot[live] // page].long() * page + slot[live] % page
        assert torch.equal(out[1][:9000].cpu()[live], at) and bool((out[1][:9000].cpu()[~live] == -1).all())
