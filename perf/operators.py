"""Cases and plain forms of the paged-cache operators.

Five operators share one key/value cache kept in pages (k, v: [n_pages, page_size, H_kv, d] bf16; block_table:
[n_seq, max_blocks] int32; seq_lens: [n_seq] int32; weights, positions: [n_pages, H_kv, page_size]):

  append   the new tokens' rows of k and v go into the pages, with weight 0 and their position
  attend   attention of a few new tokens per sequence (one, or a tree of drafted ones) over the cache and each other
  weigh    the attention weight that each cached key received is added to the weight it has gathered
  select   which keys stay when the cache shrinks to a budget: the newest and those with the most weight
  compact  the kept rows beyond the budget move into the slots of the dropped ones

`run` computes them in plain torch operations, or, where `own` is true, by the framework's calls.
"""

import math

import numpy as np
import torch

own = False


def listed():
    return [
        # One user, one token, a short chat: latency alone.
        {"name": "attend_one_short", "op": "attend", "n_seq": 1, "longest": 1003, "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "ragged": False},
        # Token by token for a full batch of chats of different lengths: the step of a serving loop.
        {"name": "attend_batch", "op": "attend", "n_seq": 64, "longest": 8191, "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "ragged": True},
        # Verification of drafted trees of up to 60 tokens for a medium batch.
        {"name": "attend_tree", "op": "attend", "n_seq": 16, "longest": 4096, "tokens": 60, "heads": 32, "kv_heads": 8, "dim": 128, "page": 32, "ragged": True},
        # One long document, a short draft, few shared heads: the work has to be split along the keys.
        {"name": "attend_long_d64", "op": "attend", "n_seq": 1, "longest": 131072, "tokens": 5, "heads": 16, "kv_heads": 2, "dim": 64, "page": 128, "ragged": False},
        # The weights of one decoded token per sequence.
        {"name": "weigh_batch", "op": "weigh", "n_seq": 32, "longest": 8191, "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "ragged": True},
        # The weights that a whole prompt leaves behind, before the first eviction.
        {"name": "weigh_prompt", "op": "weigh", "n_seq": 1, "longest": 8000, "tokens": 8000, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "ragged": False},
        # A small cache that has run a page over its budget.
        {"name": "select_small", "op": "select", "n_seq": 2, "longest": 1040, "heads": 16, "kv_heads": 4, "page": 16, "budget": 1024, "recent": 128, "ragged": False},
        # Long prompts cut to an eighth.
        {"name": "select_long", "op": "select", "n_seq": 16, "longest": 32768, "heads": 32, "kv_heads": 8, "page": 64, "budget": 4096, "recent": 512, "ragged": True},
        # The few rows that move in a cache that has run a page over its budget.
        {"name": "compact_small", "op": "compact", "n_seq": 2, "longest": 1040, "heads": 16, "kv_heads": 4, "dim": 64, "page": 16, "budget": 1024, "ragged": False},
        # The rows that move when long prompts are cut to a quarter.
        {"name": "compact_long", "op": "compact", "n_seq": 32, "longest": 16384, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "budget": 4096, "ragged": True},
        # One decoded token per sequence.
        {"name": "append_step", "op": "append", "n_seq": 16, "longest": 2048, "tokens": 1, "heads": 16, "kv_heads": 16, "dim": 64, "page": 16, "ragged": True},
        # Whole prompts go into the cache.
        {"name": "append_prompt", "op": "append", "n_seq": 8, "longest": 4999, "tokens": 4999, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "weigh", "weigh", "select", "compact", "append"])
    kv = rng.choice([1, 2, 4, 8])
    case = {"op": op, "kv_heads": kv, "heads": kv * rng.choice([1, 2, 3, 4, 7, 8]), "page": rng.choice([16, 32, 64, 128, 48]), "ragged": rng.random() < 0.7}
    if op == "attend":
        n, tokens = _log(rng, 1, 64), rng.choice([1, 1, 2, 5, 17, 33, 60, 64, 128])
        room = min(131072, 320000 // n // max(1, tokens * case["heads"] // 256))
        case.update(n_seq=n, tokens=tokens, longest=_log(rng, min(50, room), room), dim=rng.choice([64, 128]))
    elif op == "weigh":
        if rng.random() < 0.5:
            n = _log(rng, 1, 32)
            case.update(n_seq=n, tokens=rng.choice([1, 1, 3, 8, 32]), longest=_log(rng, 50, 32 * 8192 // n // 4), dim=rng.choice([64, 128]))
        else:
            case.update(n_seq=1, tokens=0, longest=_log(rng, 130, 4000), dim=rng.choice([64, 128]))
            case["tokens"] = case["longest"]
    elif op == "append":
        n = _log(rng, 1, 64)
        case.update(n_seq=n, tokens=rng.choice([1, 1, 4, _log(rng, 2, 16000 // n)]), dim=rng.choice([64, 128]))
        case["longest"] = case["tokens"] + rng.choice([0, 0, 1, 700])
    else:
        n = _log(rng, 1, 32)
        longest = _log(rng, 200, min(65536, 16 * 16384 // n))
        case.update(n_seq=n, longest=longest, budget=max(16, int(longest * rng.choice([0.9, 0.5, 0.25, 0.1]))))
        if op == "select":
            case["recent"] = rng.choice([0, 1, case["budget"] // 8, case["budget"] // 2])
        else:
            case["dim"] = rng.choice([64, 128])
    return case


# ------------------------------------------------------------------ shapes


def _lens(case):
    """Cached tokens of each sequence (with the new ones, where the operator comes after they were appended)."""
    n, longest = case["n_seq"], case["longest"]
    lens = [longest if i == 0 or not case["ragged"] else max(1, int(longest * (0.3 + 0.7 * ((i * 0.6180339887) % 1.0)))) for i in range(n)]
    if case["op"] in ("weigh", "append"):  # a sequence holds its new tokens at least
        lens = [max(a, t) for a, t in zip(lens, _tokens(case))]
    return lens


def _tokens(case):
    """New tokens of each sequence."""
    n, most = case["n_seq"], case["tokens"]
    return [most if i == 0 or not case["ragged"] else max(1, int(most * (0.5 + 0.5 * ((i * 0.4142135624) % 1.0)))) for i in range(n)]


def work(case):
    lens, hkv, h = _lens(case), case["kv_heads"], case["heads"]
    if case["op"] == "select":
        # weights and positions of every token in, the old slot of every kept one out; a comparison per token
        n = sum(lens)
        return {"bytes": hkv * (8 * n + 4 * len(lens) * case["budget"]), "flops": hkv * n}
    d = case["dim"]
    if case["op"] == "compact":
        # the list in; a row that moves is read and written. How many move depends on the weights: those kept beyond the budget, in proportion
        moved = sum(hkv * case["budget"] * (1 - case["budget"] / n) for n in lens if n > case["budget"])
        return {"bytes": moved * 2 * (2 * 2 * d + 8) + 4 * hkv * case["budget"] * len(lens), "flops": 0}
    new = _tokens(case)
    if case["op"] == "append":
        return {"bytes": sum(new) * hkv * (2 * 2 * 2 * d + 8), "flops": 0}
    if case["op"] == "attend":
        keys = sum(a + t for a, t in zip(lens, new))
        rows = sum(new)
        return {"bytes": 4 * keys * hkv * d + rows * h * (4 * d + 4), "flops": 4 * h * d * sum(t * (a + (t + 1) / 2) for a, t in zip(lens, new))}
    keys, rows = sum(lens), sum(new)
    return {"bytes": keys * hkv * (2 * d + 8) + rows * h * (2 * d + 4), "flops": 2 * h * d * sum(t * (a - (t - 1) / 2) for a, t in zip(lens, new))}


# ------------------------------------------------------------------ inputs


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    n, hkv, page, h = case["n_seq"], case["kv_heads"], case["page"], case["heads"]
    lens = _lens(case)
    blocks = max(-(-a // page) for a in lens)
    n_pages = n * blocks + 3  # pages of finished requests lie between
    table = torch.randperm(n_pages, generator=g, device="cuda")[: n * blocks].view(n, blocks).to(torch.int32)
    s = {"case": case, "block_table": table, "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "max_len": max(lens)}
    if "dim" in case:
        d = case["dim"]
        s["k"] = _rand(g, n_pages, page, hkv, d).bfloat16()
        s["v"] = _rand(g, n_pages, page, hkv, d).bfloat16()
    if case["op"] in ("weigh", "select", "compact", "append"):
        # gathered weights: heavy-tailed, and exactly 0 for tokens that nothing looked at yet (ties)
        w = torch.exp(2.0 * _rand(g, n_pages, hkv, page))
        s["weights"] = w * (torch.rand(w.shape, generator=g, device="cuda") > 0.1)
        # positions: as many tokens again were evicted before, so they run ahead of the slots, out of order
        s["seq_pos"] = s["seq_lens"] * 2
        ends = torch.ones(n_pages, device="cuda", dtype=torch.float64)
        ends[table.long()] = s["seq_pos"].double()[:, None]
        s["positions"] = (torch.rand(w.shape, generator=g, device="cuda").double() * ends[:, None, None]).to(torch.int32)
    if "tokens" in case:
        new = _tokens(case)
        s["cu"] = torch.tensor([0] + np.cumsum(new).tolist(), dtype=torch.int32, device="cuda")
        s["max_new"] = max(new)
        total = sum(new)
    if case["op"] in ("attend", "append"):
        s["k_new"] = _rand(g, total, hkv, d).bfloat16()
        s["v_new"] = _rand(g, total, hkv, d).bfloat16()
    if case["op"] == "attend":
        s["q"] = (1.5 * _rand(g, total, h, d)).bfloat16()
        at = torch.cat([torch.arange(t) for t in new]).cuda()  # a token's place in its tree
        back = torch.rand(total, generator=g, device="cuda") ** 2 * 4
        s["parents"] = torch.clamp(at - 1 - back.to(torch.int64), min=-1).to(torch.int32)
    if case["op"] == "weigh":
        s["q"] = (1.5 * _rand(g, total, h, d)).bfloat16()
        s["lse"] = _lse(s)
        s["out"] = torch.zeros_like(s["weights"])
    if case["op"] == "compact":
        s["kept"] = _kept(_keys(s, 0), s["seq_lens"], case["budget"])
    return s


# ------------------------------------------------------------------ the operators, plainly


def _slots(s):
    """Page and place in it of every slot of the longest sequence: [n_seq, max_len]."""
    j = torch.arange(s["max_len"], device="cuda")
    page = s["case"]["page"]
    return s["block_table"].long()[:, j // page], (j % page).expand(s["block_table"].shape[0], -1)


def _padded(s):
    """Packed row of each sequence's token, [n_seq, max_new], and whether there is one."""
    t = torch.arange(s["max_new"], device="cuda")
    cu = s["cu"].long()
    there = t < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + t, 0), there


def _packed(x, s):
    """[n_seq, max_new, ...] -> [total, ...]"""
    return x[_padded(s)[1]]


def _attend(s):
    case = s["case"]
    hkv, d = case["kv_heads"], case["dim"]
    page, place = _slots(s)
    rows, there = _padded(s)
    n, t = rows.shape
    # keys: the cache's, then the new tokens'
    k = torch.cat([s["k"][page, place].float(), s["k_new"][rows].float()], 1)
    v = torch.cat([s["v"][page, place].float(), s["v_new"][rows].float()], 1)
    q = s["q"][rows].float().view(n, t, hkv, -1, d)
    # a token sees its ancestors: the closure of the parents' relation, doubled seven times for trees of up to 128
    up = (s["parents"].long()[rows][:, :, None] == torch.arange(t, device="cuda")).float()
    up = torch.clamp(up + torch.eye(t, device="cuda"), max=1)
    for _ in range(7):
        up = torch.clamp(up @ up, max=1)
    old = (torch.arange(page.shape[1], device="cuda") < s["seq_lens"][:, None])[:, None, :].expand(n, t, -1)
    seen = torch.cat([old, (up > 0) & there[:, None, :]], 2)
    z = torch.einsum("bthgd,blhd->bhgtl", q, k) / math.sqrt(d)
    z = torch.where(seen[:, None, None], z, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(torch.cat([old[:, 0], there], 1)[:, :, None, None], v, 0)
    o = torch.einsum("bhgtl,blhd->bthgd", p / total, v)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(n, t, -1)
    return _packed(o.reshape(n, t, -1, d), s).bfloat16(), _packed(lse, s).t().contiguous()


def _scores(s):
    """Scores of the packed queries, [n_seq, hkv, group, max_new, max_len], -inf where a query does not see a key."""
    case = s["case"]
    page, place = _slots(s)
    rows, there = _padded(s)
    n, t = rows.shape
    k = s["k"][page, place].float()
    q = s["q"][rows].float().view(n, t, case["kv_heads"], -1, case["dim"])
    new = (s["cu"][1:] - s["cu"][:-1])[:, None, None]
    last = s["seq_lens"][:, None, None] - new + torch.arange(t, device="cuda")[:, None]
    seen = (torch.arange(page.shape[1], device="cuda") <= last) & there[:, :, None]
    z = torch.einsum("bthgd,blhd->bhgtl", q, k) / math.sqrt(case["dim"])
    return z.masked_fill_(~seen[:, None, None], -math.inf)


def _lse(s):
    lse = torch.logsumexp(_scores(s), -1)  # [n, hkv, g, t]
    n, t = lse.shape[0], lse.shape[3]
    return _packed(lse.permute(0, 3, 1, 2).reshape(n, t, -1), s).t().contiguous()


def _weigh(s):
    z = _scores(s)
    rows, there = _padded(s)
    n, hkv, group, t, length = z.shape
    lse = s["lse"].t()[rows].view(n, t, hkv, group).permute(0, 2, 3, 1)
    p = torch.exp(z - lse[..., None]).sum((2, 3))  # [n, hkv, length]
    page, place = _slots(s)
    live = torch.arange(length, device="cuda") < s["seq_lens"][:, None]
    page, place = page[live], place[live]
    out = s["out"]
    out[page, :, place] = s["weights"][page, :, place] + p.permute(0, 2, 1)[live]
    return out


def _keys(s, recent):
    """What the slots are ranked by, [n_seq, hkv, max_len]: the newest tokens before all others."""
    page, place = _slots(s)
    w = s["weights"][page, :, place].permute(0, 2, 1)
    pos = s["positions"][page, :, place].permute(0, 2, 1)
    return torch.where(pos >= (s["seq_pos"] - recent)[:, None, None], math.inf, w)


def _kept(key, seq_lens, budget):
    """Old slot of the token that is at each slot afterwards, [n_seq, hkv, budget]; -1 behind the last."""
    n, hkv, length = key.shape
    if length < budget:
        key = torch.nn.functional.pad(key, (0, budget - length), value=-math.inf)
        length = budget
    slot = torch.arange(length, device=key.device)
    live = slot < seq_lens[:, None, None]
    order = torch.sort(torch.where(live, key, -math.inf), dim=-1, descending=True, stable=True)[1][..., :budget]
    keep = torch.zeros(n, hkv, length, dtype=torch.bool, device=key.device).scatter_(2, order, True) & live
    below = torch.clamp(seq_lens, max=budget)[:, None, None]
    moves = keep & (slot >= below)
    sources = torch.sort(torch.where(moves, slot, length), dim=-1)[0][..., :budget]
    hole = ~keep[..., :budget]
    rank = torch.clamp(torch.cumsum(hole, -1) - 1, min=0)
    kept = torch.where(hole, sources.gather(2, rank), slot[:budget])
    return torch.where(slot[:budget] < below, kept, -1).to(torch.int32)


def _compact(s):
    kept, budget, page = s["kept"], s["case"]["budget"], s["case"]["page"]
    b, h, to = torch.nonzero(kept >= budget, as_tuple=True)
    frm = kept[b, h, to].long()
    pf, jf = s["block_table"][b, frm // page].long(), frm % page
    pt, jt = s["block_table"][b, to // page].long(), to % page
    s["k"][pt, jt, h] = s["k"][pf, jf, h]
    s["v"][pt, jt, h] = s["v"][pf, jf, h]
    s["weights"][pt, h, jt] = s["weights"][pf, h, jf]
    s["positions"][pt, h, jt] = s["positions"][pf, h, jf]
    return s["k"], s["v"], s["weights"], s["positions"]


def _append(s):
    page, t = s["case"]["page"], torch.arange(s["max_new"], device="cuda")
    rows, there = _padded(s)
    new = (s["cu"][1:] - s["cu"][:-1])[:, None]
    slot = (s["seq_lens"][:, None] - new + t)[there].long()
    pos = (s["seq_pos"][:, None] - new + t)[there].to(torch.int32)
    b = torch.arange(rows.shape[0], device="cuda")[:, None].expand_as(rows)[there]
    p, j = s["block_table"][b, slot // page].long(), slot % page
    s["k"][p, j] = s["k_new"]
    s["v"][p, j] = s["v_new"]
    s["weights"][p, :, j] = 0.0
    s["positions"][p, :, j] = pos[:, None]
    return s["k"], s["v"], s["weights"], s["positions"]


def run(s):
    case = s["case"]
    if own:
        from exact_attention_63_gb300 import cache

        if case["op"] == "attend":
            return cache.attn_fwd_cache(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["block_table"], s["seq_lens"], s["cu"], s["max_new"], parents=s["parents"])
        if case["op"] == "weigh":
            return cache.cache_weights(s["q"], s["lse"], s["k"], s["block_table"], s["seq_lens"], s["cu"], s["max_new"], s["weights"], out=s["out"])
        if case["op"] == "select":
            return cache.cache_select(s["weights"], s["block_table"], s["seq_lens"], case["budget"], recent=case["recent"], positions=s["positions"], seq_pos=s["seq_pos"])
        if case["op"] == "compact":
            cache.cache_compact(s["kept"], s["k"], s["v"], s["block_table"], weights=s["weights"], positions=s["positions"])
        else:
            cache.cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["block_table"], s["seq_lens"], s["cu"], weights=s["weights"], positions=s["positions"], seq_pos=s["seq_pos"])
        return s["k"], s["v"], s["weights"], s["positions"]
    if case["op"] == "attend":
        return _attend(s)
    if case["op"] == "weigh":
        return _weigh(s)
    if case["op"] == "select":
        return _kept(_keys(s, case["recent"]), s["seq_lens"], case["budget"])
    return _compact(s) if case["op"] == "compact" else _append(s)


# ------------------------------------------------------------------ the definition in 64 bits


def _one(s, b, x):
    """Sequence b's rows of paged x, in slot order."""
    n = int(s["seq_lens"][b])
    page = s["case"]["page"]
    used = s["block_table"][b, : -(-n // page)].long()
    if x.dim() == 3:  # [pages, hkv, page] -> [n, hkv]
        x = x.transpose(1, 2)
    return x[used].flatten(0, 1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    n, hkv, op = case["n_seq"], case["kv_heads"], case["op"]
    if op in ("compact", "append"):
        return None  # values are moved, none is computed
    if op == "select":
        kept = np.full((n, hkv, case["budget"]), -1, np.int32)
        for b in range(n):
            w = _one(s, b, s["weights"]).double().cpu().numpy()
            pos = _one(s, b, s["positions"]).cpu().numpy()
            newest = pos >= int(s["seq_pos"][b]) - case["recent"]
            for h in range(hkv):
                order = np.lexsort((np.arange(len(w)), -w[:, h], ~newest[:, h]))[: case["budget"]]
                m = min(len(w), case["budget"])
                stay, move = order[order < m], np.sort(order[order >= m])
                row = np.full(m, -1, np.int32)
                row[stay] = stay
                row[row < 0] = move
                kept[b, h, :m] = row
        return torch.from_numpy(kept)
    cu = s["cu"].tolist()
    group, scale = case["heads"] // hkv, 1.0 / math.sqrt(case["dim"])
    if op == "attend":
        total = cu[-1]
        o = torch.empty(total, case["heads"], case["dim"], dtype=torch.float64, device="cuda")
        lse = torch.empty(case["heads"], total, dtype=torch.float64, device="cuda")
        parents = s["parents"].tolist()
        for b in range(n):
            rows, length = slice(cu[b], cu[b + 1]), int(s["seq_lens"][b])
            t = cu[b + 1] - cu[b]
            seen = np.zeros((t, t), bool)
            for i in range(t):
                j = i
                while j >= 0:
                    seen[i, j] = True
                    j = parents[cu[b] + j]
            hide = torch.cat([torch.zeros(t, length, dtype=torch.bool), torch.from_numpy(~seen)], 1).cuda()
            k = torch.cat([_one(s, b, s["k"]), s["k_new"][rows]]).double()
            v = torch.cat([_one(s, b, s["v"]), s["v_new"][rows]]).double()
            for h in range(hkv):
                q = s["q"][rows, h * group : (h + 1) * group].double().transpose(0, 1)  # [g, t, d]
                z = (q @ k[:, h].t() * scale).masked_fill(hide, -math.inf)
                l = torch.logsumexp(z, -1)
                o[rows, h * group : (h + 1) * group] = (torch.exp(z - l[..., None]) @ v[:, h]).transpose(0, 1)
                lse[h * group : (h + 1) * group, rows] = l
        return o, lse
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    page = case["page"]
    for b in range(n):
        rows, length = slice(cu[b], cu[b + 1]), int(s["seq_lens"][b])
        t = cu[b + 1] - cu[b]
        k = _one(s, b, s["k"]).double()
        gathered = _one(s, b, s["weights"]).double()  # [length, hkv]
        last = length - t + torch.arange(t, device="cuda")
        for h in range(hkv):
            for m in range(group):
                z = s["q"][rows, h * group + m].double() @ k[:, h].t() * scale
                p = torch.exp(z - s["lse"][h * group + m, rows].double()[:, None])
                p[torch.arange(length, device="cuda") > last[:, None]] = 0.0
                gathered[:, h] += p.sum(0)
        j = torch.arange(length, device="cuda")
        out[s["block_table"][b].long()[j // page], :, j % page] = gathered
    return out
