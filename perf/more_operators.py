"""Cases and plain forms of the operators around a key/value cache held in 8 bits.

The cache: pages k, v [n_pages, page_size, H_kv, d] of E4M3 codes and, for every 16 slots of a page and every key head,
an exponent byte k_scales, v_scales [n_pages, H_kv, page_size / 16]: a code c stands for c * 2^(byte - 127).

  attend   attention of a few new tokens per sequence (one, or a tree of drafted ones) over the cache and each other
  append   new tokens' rows of k and v are rounded into the pages; a block that gets larger values gets a larger scale
  gather   the newest rows of each sequence, back in bf16 and packed
  rotary   rotary positions on q and k: halves or interleaved, the whole head or part of it, scaled for long contexts
  pages    block tables follow the requests' lengths: pages come from and go back to a stack, new tokens get their slots

`run` computes them in plain torch operations, or, where `own` is true, by the framework's calls.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16  # slots that share a scale
LOWEST, HIGHEST = -117, 119  # exponents of a scale


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
        # The tokens of one decoding step go into the cache.
        {"name": "append_step", "op": "append", "n_seq": 64, "longest": 8191, "tokens": 1, "kv_heads": 8, "dim": 128, "page": 64, "ragged": True},
        # Whole prompts go into the cache.
        {"name": "append_prompt", "op": "append", "n_seq": 8, "longest": 4999, "tokens": 4999, "kv_heads": 8, "dim": 128, "page": 64, "ragged": True},
        # What a prompt's next piece attends over when the pieces are longer than a draft.
        {"name": "gather_long", "op": "gather", "n_seq": 2, "longest": 32768, "tokens": 32768, "kv_heads": 8, "dim": 128, "page": 64, "ragged": True},
        # A window of the newest tokens of many short chats.
        {"name": "gather_window", "op": "gather", "n_seq": 48, "longest": 1500, "tokens": 256, "kv_heads": 4, "dim": 64, "page": 16, "ragged": True},
        # A training batch, forward and backward.
        {"name": "rotary_train", "op": "rotary", "batch": 4, "rows": 4096, "heads": 32, "kv_heads": 8, "dim": 128, "part": 128, "interleaved": False, "factor": 1.0, "far": 0, "backward": True},
        # One decoding step far into a context that is longer than the one trained on; half the head turns.
        {"name": "rotary_step", "op": "rotary", "batch": 1, "rows": 64, "heads": 32, "kv_heads": 8, "dim": 128, "part": 64, "interleaved": True, "factor": 8.0, "far": 131072, "backward": False},
        # Room for one more token of every running request, or for two, given back again.
        {"name": "pages_step", "op": "pages", "n_seq": 256, "longest": 4096, "tokens": 2, "page": 16, "ragged": True},
        # Room for new prompts.
        {"name": "pages_prompts", "op": "pages", "n_seq": 64, "longest": 8191, "tokens": 8191, "page": 16, "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "append", "append", "gather", "rotary", "rotary", "pages"])
    case = {"op": op}
    kv = rng.choice([1, 2, 4, 8])
    if op == "rotary":
        dim = rng.choice([64, 128])
        rows = _log(rng, 1, 4096)
        case.update(batch=rng.choice([1, 1, 2, 3]), rows=rows, heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv, dim=dim)
        case.update(part=rng.choice([dim, dim, dim // 2, dim // 4, 24]), interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 2.0, 8.0, 32.0]))
        case.update(far=rng.choice([0, 1, 5000, 131072, 1000003]), backward=rng.random() < 0.5)
        return case
    case.update(page=rng.choice([16, 32, 64, 128, 48]), ragged=rng.random() < 0.7)
    if op == "pages":
        n = _log(rng, 1, 512)
        case.update(n_seq=n, longest=_log(rng, 20, min(65536, 500000 // n)))
        case["tokens"] = rng.choice([1, 1, 2, 7, case["longest"]])
        return case
    case.update(kv_heads=kv, dim=rng.choice([64, 128]))
    if op == "attend":
        n, tokens = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 17, 33, 60, 64, 128])
        case["heads"] = kv * rng.choice([1, 2, 3, 4, 7, 8])
        n = min(n, max(1, 200000 // (tokens * case["heads"])))
        room = min(131072, 300000 // n // max(1, tokens * case["heads"] // 160))
        case.update(n_seq=n, tokens=tokens, longest=_log(rng, min(50, room), room))
    elif op == "append":
        n = _log(rng, 1, 64)
        case.update(n_seq=n, tokens=rng.choice([1, 1, 4, 17, _log(rng, 2, 20000 // n)]))
        case["longest"] = case["tokens"] + rng.choice([0, 1, 7, 700])
    else:
        n = _log(rng, 1, 64)
        case.update(n_seq=n, longest=_log(rng, 50, 60000 // n))
        case["tokens"] = rng.choice([case["longest"], case["longest"], 1 + case["longest"] // 3, 16])
        case["tokens"] = min(case["tokens"], case["longest"])
    return case


# ------------------------------------------------------------------ shapes


def _tokens(case):
    """New tokens of each sequence (gather: the newest ones asked for)."""
    n, most = case["n_seq"], case["tokens"]
    return [most if i == 0 or not case["ragged"] else max(1, int(most * (0.5 + 0.5 * ((i * 0.4142135624) % 1.0)))) for i in range(n)]


def _lens(case):
    """Cached tokens of each sequence (with the new ones, but for attend)."""
    n, longest = case["n_seq"], case["longest"]
    lens = [longest if i == 0 or not case["ragged"] else max(1, int(longest * (0.3 + 0.7 * ((i * 0.6180339887) % 1.0)))) for i in range(n)]
    return lens if case["op"] == "attend" else [max(a, t) for a, t in zip(lens, _tokens(case))]


def work(case):
    op = case["op"]
    if op == "rotary":
        rows = case["batch"] * case["rows"] * (case["heads"] + case["kv_heads"])
        passes = 2 if case["backward"] else 1
        return {"bytes": passes * rows * case["dim"] * 4 + case["batch"] * case["rows"] * 4, "flops": passes * rows * case["part"] * 3}
    lens, new = _lens(case), _tokens(case)
    if op == "pages":
        # lengths, counts and offsets in, lengths' verdicts out; a page that changes hands is read and written twice; slot and position of each token
        moved = sum(-(-a // case["page"]) - -(-(a - t) // case["page"]) for a, t in zip(lens, new))
        return {"bytes": 2 * 16 * len(lens) + 16 * moved + 12 * sum(new), "flops": sum(new)}
    hkv, d = case["kv_heads"], case["dim"]
    if op == "attend":
        keys, rows, h = sum(lens), sum(new), case["heads"]
        return {"bytes": hkv * (keys * 2 * d + keys / 8 + rows * 4 * d) + rows * h * (4 * d + 4), "flops": 4 * h * d * sum(t * (a + (t + 1) / 2) for a, t in zip(lens, new))}
    if op == "append":
        # rows in and out; what is read back: the newest rows of each sequence
        back = sum(_back(a, t) for a, t in zip(lens, new))
        return {"bytes": hkv * d * (sum(new) * (4 + 2) + back * (2 + 4)), "flops": 2 * hkv * d * sum(new)}
    return {"bytes": hkv * d * sum(new) * (2 + 4), "flops": 2 * hkv * d * sum(new)}


def _back(length, new):
    """Rows that a sequence's append may change: the new ones, and the older ones of the block that they begin in."""
    return new + (length - new) % BLOCK


# ------------------------------------------------------------------ inputs


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _power(e):
    """2^e of whole numbers e within fp32's normal range, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(top):
    """The smallest e with top <= 448 * 2^e, within bounds: 448 is 1.75 * 2^8."""
    bits = top.float().contiguous().view(torch.int32)
    return torch.clamp((bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000), LOWEST, HIGHEST)


def _codes(x, e):
    """x in units of 2^e (exponents that broadcast), rounded to E4M3."""
    half = torch.div(-e, 2, rounding_mode="floor")
    y = x.float() * _power(half) * _power(-e - half)
    return torch.clamp(y, -448.0, 448.0).to(torch.float8_e4m3fn)


def _filled(g, case, n_pages):
    """Pages of quantised rows, whose heads and tokens differ in size as those of a model do."""
    page, hkv, d = case["page"], case["kv_heads"], case["dim"]
    x = _rand(g, n_pages, page // BLOCK, BLOCK, hkv, d)
    x *= torch.exp(0.5 * _rand(g, 1, 1, 1, hkv, d))
    e = _exponent(x.abs().amax((2, 4), keepdim=True))
    codes = _codes(x, e).view(n_pages, page, hkv, d)
    return codes, (e[:, :, 0, :, 0].transpose(1, 2) + 127).to(torch.uint8).contiguous()


def _frequencies(case):
    """Radians a position of each pair, float64.  A factor above 1 stretches the slow ones by it, those that turn more than
    32 times in 4096 positions not at all, and those between in proportion."""
    part = case["part"]
    f = 10000.0 ** (-torch.arange(0, part, 2, dtype=torch.float64) / part)
    if case["factor"] > 1.0:
        at = [part * math.log(4096 / (b * 2 * math.pi)) / (2 * math.log(10000.0)) for b in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), part - 1)
        keep = 1.0 - torch.clamp((torch.arange(part // 2, dtype=torch.float64) - low) / max(high - low, 0.001), 0.0, 1.0)
        f = f / case["factor"] * (1.0 - keep) + f * keep
    return f


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    s = {"case": case}
    if case["op"] == "rotary":
        b, rows, d = case["batch"], case["rows"], case["dim"]
        # q and k are slices of one projection's output, as the layers before leave them
        both = _rand(g, b, rows, case["heads"] + case["kv_heads"], d).bfloat16()
        s["q"], s["k"] = both[:, :, : case["heads"]], both[:, :, case["heads"] :]
        s["dq"] = _rand(g, b, rows, case["heads"], d).bfloat16()
        s["dk"] = _rand(g, b, rows, case["kv_heads"], d).bfloat16()
        if case["far"]:  # requests at places of their own
            s["positions"] = torch.randint(0, case["far"] + 1, (b, rows), generator=g, device="cuda", dtype=torch.int32)
        else:
            s["positions"] = torch.arange(rows, device="cuda", dtype=torch.int32).expand(b, rows).contiguous()
        s["inv_freq"] = _frequencies(case).cuda()
        s["magnitude"] = 1.0 if case["factor"] <= 1.0 else 0.1 * math.log(case["factor"]) + 1.0
        return s
    n, page = case["n_seq"], case["page"]
    lens, new = _lens(case), _tokens(case)
    s["cu"] = torch.tensor([0] + np.cumsum(new).tolist(), dtype=torch.int32, device="cuda")
    s["max_new"], s["total"] = max(new), sum(new)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["max_len"] = max(lens)
    blocks = max(-(-a // page) for a in lens)
    if case["op"] == "pages":
        before = [a - t for a, t in zip(lens, new)]
        held = [-(-a // page) for a in before]
        n_pages = max(sum(held), sum(-(-a // page) for a in lens) + 3 - n // 100)  # now and then too few
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        taken = sum(held)
        there = torch.arange(blocks + 2) < torch.tensor(held)[:, None]
        s["block_table"] = torch.full((n, blocks + 2), -1, dtype=torch.int32, device="cuda")
        s["block_table"][there.cuda()] = order[:taken]
        s["free_pages"] = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        s["free_pages"][: n_pages - taken] = order[taken:]
        s["n_free"] = torch.tensor([n_pages - taken], dtype=torch.int32, device="cuda")
        s["n_blocks"] = torch.tensor(held, dtype=torch.int32, device="cuda")
        s["before"] = torch.tensor(before, dtype=torch.int32, device="cuda")
        return s
    hkv, d = case["kv_heads"], case["dim"]
    n_pages = n * blocks + 3  # pages of finished requests lie between
    s["block_table"] = torch.randperm(n_pages, generator=g, device="cuda")[: n * blocks].view(n, blocks).to(torch.int32)
    s["k"], s["k_scales"] = _filled(g, case, n_pages)
    s["v"], s["v_scales"] = _filled(g, case, n_pages)
    if case["op"] in ("attend", "append"):
        s["k_new"] = (1.3 * _rand(g, s["total"], hkv, d)).bfloat16()
        s["v_new"] = (1.3 * _rand(g, s["total"], hkv, d)).bfloat16()
    if case["op"] == "attend":
        s["q"] = (1.5 * _rand(g, s["total"], case["heads"], d)).bfloat16()
        at = torch.cat([torch.arange(t) for t in new]).cuda()  # a token's place in its tree
        back = torch.rand(s["total"], generator=g, device="cuda") ** 2 * 4
        s["parents"] = torch.clamp(at - 1 - back.to(torch.int64), min=-1).to(torch.int32)
    if case["op"] == "append":
        back = [_back(a, t) for a, t in zip(lens, new)]
        s["cu_back"] = torch.tensor([0] + np.cumsum(back).tolist(), dtype=torch.int32, device="cuda")
        s["max_back"], s["total_back"] = max(back), sum(back)
    return s


# ------------------------------------------------------------------ the operators, plainly


def _padded(cu, most):
    """Packed row of each sequence's token, [n_seq, most], and whether there is one."""
    t = torch.arange(most, device="cuda")
    cu = cu.long()
    there = t < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + t, 0), there


def _values(codes, scales, page, place):
    """What the slots stand for, fp32 [..., hkv, d]; page and place of the slots: [...]."""
    x = codes.view(torch.uint8)[page, place].view(torch.float8_e4m3fn).float()
    return x * _power(scales[page, :, place // BLOCK].to(torch.int32) - 127)[..., None]


def _attend(s):
    case = s["case"]
    hkv, d, page = case["kv_heads"], case["dim"], case["page"]
    j = torch.arange(s["max_len"], device="cuda")
    rows, there = _padded(s["cu"], s["max_new"])
    n, t = rows.shape
    at, place = s["block_table"].long()[:, j // page], (j % page).expand(n, -1)
    # keys: the cache's, then the new tokens'
    k = torch.cat([_values(s["k"], s["k_scales"], at, place), s["k_new"][rows].float()], 1)
    v = torch.cat([_values(s["v"], s["v_scales"], at, place), s["v_new"][rows].float()], 1)
    q = s["q"][rows].float().view(n, t, hkv, -1, d)
    # a token sees its ancestors: the closure of the parents' relation, doubled seven times for trees of up to 128
    up = (s["parents"].long()[rows][:, :, None] == torch.arange(t, device="cuda")).float()
    up = torch.clamp(up + torch.eye(t, device="cuda"), max=1)
    up = torch.clamp(up @ up, max=1)
    up = torch.clamp(up @ up, max=1)
    up = torch.clamp(up @ up, max=1)
    up = torch.clamp(up @ up, max=1)
    up = torch.clamp(up @ up, max=1)
    up = torch.clamp(up @ up, max=1)
    up = torch.clamp(up @ up, max=1)
    old = (j < s["seq_lens"][:, None])[:, None, :].expand(n, t, -1)
    seen = torch.cat([old, (up > 0) & there[:, None, :]], 2)
    z = torch.einsum("bthgd,blhd->bhgtl", q, k) / math.sqrt(d)
    z = torch.where(seen[:, None, None], z, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(torch.cat([old[:, 0], there], 1)[:, :, None, None], v, 0)
    o = torch.einsum("bhgtl,blhd->bthgd", p / total, v)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(n, t, -1)
    return o.reshape(n, t, -1, d)[there].bfloat16(), lse[there].t().contiguous()


def _newest(s, cu, most):
    """Page and place of the newest slots of each sequence, in the packed order of `cu`."""
    page = s["case"]["page"]
    _, there = _padded(cu, most)
    slot = (s["seq_lens"] - (cu[1:] - cu[:-1]))[:, None] + torch.arange(most, device="cuda")
    b = torch.arange(there.shape[0], device="cuda")[:, None].expand_as(there)[there]
    slot = slot[there].long()
    return b, slot, s["block_table"][b, slot // page].long(), slot % page


def _read(s, cu, most):
    _, _, page, place = _newest(s, cu, most)
    return _values(s["k"], s["k_scales"], page, place).bfloat16(), _values(s["v"], s["v_scales"], page, place).bfloat16()


def _put(s, codes, scales, new):
    """The rows `new` go into the pages of codes and scales."""
    case = s["case"]
    size, hkv = case["page"], case["kv_heads"]
    b, slot, page, place = _newest(s, s["cu"], s["max_new"])
    block, per = slot // BLOCK, size // BLOCK
    # the blocks that get rows, by a number of their own: their largest new value, and whether older rows stay in them
    most = int(s["max_len"] // BLOCK + 1)
    key = b * most + block
    top = torch.zeros(s["seq_lens"].shape[0] * most, hkv, device="cuda")
    x = new.float()
    top.index_reduce_(0, key, torch.where(torch.isfinite(x), x.abs(), 0).amax(-1), "amax")
    first = (s["seq_lens"] - (s["cu"][1:] - s["cu"][:-1]))[b]
    kept = block * BLOCK < first
    e_new = _exponent(top[key])  # [rows, hkv]
    e_old = scales[page, :, place // BLOCK].to(torch.int32) - 127
    e = torch.where(kept[:, None], torch.maximum(e_new, e_old), e_new)
    # older rows of a block whose scale grows: all 16 rows in new units (the new rows are written over it)
    opens = kept & (slot == first)
    grow = torch.clamp((e_old - e)[opens], min=-126)
    at, rows = page[opens][:, None], (place[opens] // BLOCK * BLOCK)[:, None] + torch.arange(BLOCK, device="cuda")
    old = codes.view(torch.uint8)[at, rows].view(torch.float8_e4m3fn).float()
    codes.view(torch.uint8)[at, rows] = (old * _power(grow)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes.view(torch.uint8)[page, place] = _codes(x, e[:, :, None]).view(torch.uint8)
    scales.view(-1, hkv, per)[page, :, place // BLOCK] = (e + 127).to(torch.uint8)


def _append(s):
    _put(s, s["k"], s["k_scales"], s["k_new"])
    _put(s, s["v"], s["v_scales"], s["v_new"])
    return _read(s, s["cu_back"], s["max_back"])


def _turned(s, x, sign):
    case = s["case"]
    part = case["part"]
    angle = s["positions"].double()[..., None, None] * s["inv_freq"]
    c, n = (torch.cos(angle) * s["magnitude"]).float(), (sign * torch.sin(angle) * s["magnitude"]).float()
    y = x[..., :part].float()
    if case["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = y[..., : part // 2], y[..., part // 2 :]
        y = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([y.bfloat16(), x[..., part:]], -1)


def _rotary(s):
    out = [_turned(s, s["q"], 1.0), _turned(s, s["k"], 1.0)]
    if s["case"]["backward"]:
        out += [_turned(s, s["dq"], -1.0), _turned(s, s["dk"], -1.0)]
    return out


def _resize(s, lens):
    """The tables hold room for `lens` tokens afterwards, where there are pages; pages that each sequence lacked."""
    page, table, free = s["case"]["page"], s["block_table"], s["free_pages"]
    want = (lens + page - 1) // page
    held, j = s["n_blocks"].clone(), torch.arange(table.shape[1], device="cuda", dtype=torch.int32)
    drop = (j >= want[:, None]) & (j < held[:, None])
    rank = torch.cumsum(drop.flatten(), 0).view_as(drop) - 1
    free[(s["n_free"] + rank)[drop]] = table[drop]
    table[drop] = -1
    s["n_free"] += drop.sum().to(torch.int32)
    held = torch.minimum(held, want)
    wide = want > table.shape[1]
    need = torch.where(wide, 0, want - held)
    through = torch.cumsum(need, 0)
    served = ((need == 0) | (through <= s["n_free"])) & ~wide
    got = (j >= held[:, None]) & (j < want[:, None]) & served[:, None]
    rank = (through - need)[:, None] + j - held[:, None]
    table[got] = free[(s["n_free"] - 1 - rank)[got].long()]
    s["n_free"] -= got.sum().to(torch.int32)
    s["n_blocks"].copy_(torch.where(served, want, held))
    return torch.where(served, 0, want - held).to(torch.int32)


def _pages(s):
    missing = _resize(s, s["seq_lens"])
    page = s["case"]["page"]
    b, slot, at, place = _newest(s, s["cu"], s["max_new"])
    slots = torch.where((missing == 0)[b], at * page + place, -1)
    _resize(s, s["before"])  # the tokens are not taken: their pages go back
    return missing, slots, slot.to(torch.int32), s["block_table"], s["n_blocks"], s["free_pages"], s["n_free"]


def run(s):
    case = s["case"]
    if own:
        from exact_attention_63_gb300 import cache, rotary

        if case["op"] == "attend":
            return cache.attn_fwd_cache_fp8(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["k_scales"], s["v_scales"], s["block_table"], s["seq_lens"], s["cu"], s["max_new"], parents=s["parents"])
        if case["op"] == "append":
            cache.cache_append_fp8(s["k_new"], s["v_new"], s["k"], s["v"], s["k_scales"], s["v_scales"], s["block_table"], s["seq_lens"], s["cu"])
            return cache.cache_gather_fp8(s["k"], s["v"], s["k_scales"], s["v_scales"], s["block_table"], s["seq_lens"], s["cu_back"], s["total_back"])
        if case["op"] == "gather":
            return cache.cache_gather_fp8(s["k"], s["v"], s["k_scales"], s["v_scales"], s["block_table"], s["seq_lens"], s["cu"], s["total"])
        if case["op"] == "pages":
            missing, slots, positions = cache.cache_pages(s["seq_lens"], s["block_table"], s["n_blocks"], s["free_pages"], s["n_free"], case["page"], cu_new=s["cu"], total=s["total"])
            cache.cache_pages(s["before"], s["block_table"], s["n_blocks"], s["free_pages"], s["n_free"], case["page"])
            return missing, slots, positions, s["block_table"], s["n_blocks"], s["free_pages"], s["n_free"]
        out = rotary.rotary_fwd(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=case["interleaved"], magnitude=s["magnitude"])
        if case["backward"]:
            out += rotary.rotary_bwd(s["dq"], s["dk"], s["positions"], s["inv_freq"], interleaved=case["interleaved"], magnitude=s["magnitude"])
        return out
    if case["op"] == "attend":
        return _attend(s)
    if case["op"] == "append":
        return _append(s)
    if case["op"] == "gather":
        return _read(s, s["cu"], s["max_new"])
    return _pages(s) if case["op"] == "pages" else _rotary(s)


# ------------------------------------------------------------------ the definition in 64 bits


def _decoded():
    """The 256 values of E4M3: sign, four bits of exponent with bias 7, three of fraction; NaN where all seven are set."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = math.nan if c & 127 == 127 else (-x if c & 128 else x)
    return out


def _rounded(y):
    """y to the nearest value of E4M3, ties to the even fraction; beyond the largest, the largest."""
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -20))), -6.0) - 3.0)
    return np.clip(np.rint(y / step) * step, -448.0, 448.0)


def _one(s, b, name):
    """Sequence b's rows of k or v in float64, slot by slot, on the GPU."""
    n, page = int(s["seq_lens"][b]), s["case"]["page"]
    used = s["block_table"][b, : -(-n // page)].long()
    x = torch.from_numpy(_decoded()).cuda()[s[name].view(torch.uint8)[used].long()]
    e = s[name + "_scales"][used].double().transpose(1, 2).repeat_interleave(BLOCK, 1)[..., None] - 127.0
    return (x * torch.exp2(e)).flatten(0, 1)[:n]


def _exact_append(s, name, b, t):
    """Sequence b's newest rows after its t new ones went in."""
    n, page = int(s["seq_lens"][b]), s["case"]["page"]
    new = s[name + "_new"][int(s["cu"][b]) : int(s["cu"][b + 1])].double().cpu().numpy()
    start = n - _back(n, t)
    used = s["block_table"][b].cpu().numpy()
    codes, scales = s[name].view(torch.uint8), s[name + "_scales"]
    out = np.empty((n - start,) + new.shape[1:])
    for at in range(start, n, BLOCK):
        first, last = max(at, n - t), min(at + BLOCK, n)
        x = new[first - (n - t) : last - (n - t)]
        top = np.abs(x).max((0, 2))
        e = np.empty(top.shape)
        for h, a in enumerate(top):  # the smallest power of two that holds a / 448
            m, p = math.frexp(a / 448.0)
            e[h] = min(max(p - 1 if m == 0.5 else p, LOWEST), HIGHEST) if a > 0 else LOWEST
        if first > at:
            p, j = int(used[at // page]), at % page
            old = _decoded()[codes[p, j : j + first - at].cpu().numpy()]
            e_old = scales[p, :, j // BLOCK].double().cpu().numpy() - 127.0
            e = np.maximum(e, e_old)
            out[at - start : first - start] = _rounded(old * np.exp2(e_old - e)[:, None]) * np.exp2(e)[:, None]
        out[first - start : last - start] = _rounded(x * np.exp2(-e)[:, None]) * np.exp2(e)[:, None]
    return torch.from_numpy(out)


def _exact_pages(s):
    page = s["case"]["page"]
    table, held = s["block_table"].tolist(), s["n_blocks"].tolist()
    free, top = s["free_pages"].tolist(), int(s["n_free"])
    cu, missing, slots, positions = s["cu"].tolist(), [], [], []

    def resize(lens):
        nonlocal top
        lack = []
        for row, n in zip(range(len(lens)), lens):
            want = -(-n // page)
            for j in range(want, held[row]):
                free[top] = table[row][j]
                top += 1
                table[row][j] = -1
            held[row] = min(held[row], want)
        asked, there = 0, top
        for row, n in zip(range(len(lens)), lens):
            want = -(-n // page)
            need = want - held[row]
            if want <= len(table[row]):
                asked += need
                if need and asked <= there:
                    for j in range(held[row], want):
                        top -= 1
                        table[row][j] = free[top]
                    held[row] = want
            lack.append(want - held[row])
        return lack

    lens = s["seq_lens"].tolist()
    missing = resize(lens)
    for b, n in enumerate(lens):
        for j in range(n - (cu[b + 1] - cu[b]), n):
            slots.append(-1 if missing[b] else table[b][j // page] * page + j % page)
            positions.append(j)
    resize(s["before"].tolist())
    ints = [torch.tensor(x, dtype=torch.int32) for x in (missing, positions, table, held, free, [top])]
    return ints[0], torch.tensor(slots, dtype=torch.int64), *ints[1:]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "pages":
        return _exact_pages(s)
    if op == "rotary":
        at = s["positions"].cpu().numpy().astype(np.float64)[:, :, None]
        turn = np.exp(1j * at * s["inv_freq"].cpu().numpy())[:, :, None] * s["magnitude"]
        out = []
        for name, back in (("q", False), ("k", False), ("dq", True), ("dk", True)):
            if back and not case["backward"]:
                continue
            x, half = s[name].double().cpu().numpy(), case["part"] // 2
            y = x.copy()
            a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
            z = (x[..., a] + 1j * x[..., b]) * (np.conj(turn) if back else turn)
            y[..., a], y[..., b] = z.real, z.imag
            out.append(torch.from_numpy(y))
        return out
    n, cu = case["n_seq"], s["cu"].tolist()
    if op == "append":
        return tuple(torch.cat([_exact_append(s, x, b, cu[b + 1] - cu[b]) for b in range(n)]) for x in ("k", "v"))
    if op == "gather":
        return tuple(torch.cat([_one(s, b, x)[int(s["seq_lens"][b]) - (cu[b + 1] - cu[b]) :] for b in range(n)]) for x in ("k", "v"))
    hkv, group, scale = case["kv_heads"], case["heads"] // case["kv_heads"], 1.0 / math.sqrt(case["dim"])
    o = torch.empty(cu[-1], case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.empty(case["heads"], cu[-1], dtype=torch.float64, device="cuda")
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
        k = torch.cat([_one(s, b, "k"), s["k_new"][rows].double()])
        v = torch.cat([_one(s, b, "v"), s["v_new"][rows].double()])
        for h in range(hkv):
            q = s["q"][rows, h * group : (h + 1) * group].double().transpose(0, 1)  # [g, t, d]
            z = (q @ k[:, h].t() * scale).masked_fill(hide, -math.inf)
            l = torch.logsumexp(z, -1)
            o[rows, h * group : (h + 1) * group] = (torch.exp(z - l[..., None]) @ v[:, h]).transpose(0, 1)
            lse[h * group : (h + 1) * group, rows] = l
    return o, lse
