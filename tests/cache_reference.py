"""Plain float64 definitions of the cache operators, and seeded caches for the
tests: one sequence, head and row at a time, from the operators' formulas alone."""

from __future__ import annotations

import numpy as np
import torch

HALF_BF16 = 2.0 ** -8    # the most that a rounding to bf16 is off, relative
HALF_F32 = 2.0 ** -24


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Case:
    """A cache in shuffled pages whose unused slots hold NaN, and new tokens."""

    def __init__(self, lens, new, H, hkv, d, page, seed=0, tree="random", sigma=1.0, slack=2, room=0):
        g = torch.Generator().manual_seed(seed)
        self.H, self.hkv, self.d, self.page = H, hkv, d, page
        self.lens, self.new = list(lens), list(new)
        n = len(lens)
        blocks = max(1, max(-(-(a + room) // page) for a in lens))
        used = [-(-(a + room) // page) for a in lens]
        self.n_pages = sum(used) + slack
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = torch.full((n, blocks), -1, dtype=torch.int32)
        for s in range(n):
            for b in range(used[s]):
                self.table[s, b] = order.pop()
        shape = (self.n_pages, page, hkv, d)
        self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        self.v = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        self.weights = torch.full((self.n_pages, hkv, page), float("nan"))
        self.positions = torch.full((self.n_pages, hkv, page), -7, dtype=torch.int32)
        for s in range(n):
            for j in range(lens[s]):
                p, i = int(self.table[s, j // page]), j % page
                self.k[p, i] = torch.randn((hkv, d), generator=g).bfloat16()
                self.v[p, i] = torch.randn((hkv, d), generator=g).bfloat16()
                self.weights[p, :, i] = torch.rand(hkv, generator=g) * 4
                self.positions[p, :, i] = j
        self.seq_lens = torch.tensor(lens, dtype=torch.int32)
        total = sum(new)
        self.total = total
        self.cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.q = (torch.randn((total, H, d), generator=g) * sigma).bfloat16()
        self.k_new = torch.randn((total, hkv, d), generator=g).bfloat16()
        self.v_new = torch.randn((total, hkv, d), generator=g).bfloat16()
        self.parents = None
        if tree != "chain":
            par = []
            for t in new:
                for i in range(t):
                    if tree == "random":
                        par.append(int(torch.randint(-1, i, (1,), generator=g)) if i else -1)
                    elif tree == "roots":
                        par.append(-1)
                    else:  # "line": the chain, given
                        par.append(i - 1)
            self.parents = torch.tensor(par, dtype=torch.int32)
        self.scale = d ** -0.5

    def cuda(self):
        for name in ("table", "k", "v", "weights", "positions", "seq_lens", "cu", "q", "k_new", "v_new", "parents"):
            t = getattr(self, name)
            if t is not None:
                setattr(self, name, t.cuda())
        return self

    def max_new(self):
        return max(self.new)


def rows_of(x, table, s, n):
    """Slots [0, n) of sequence s of paged x, [n, ...] (page-major [page, slot, ...])."""
    page = x.shape[1]
    return np.stack([x[int(table[s, j // page]), j % page] for j in range(n)]) if n else np.zeros((0,) + x.shape[2:])


def ancestors(parents, t):
    """[t, t] bool: which new tokens each one sees.  parents None: a chain."""
    seen = np.zeros((t, t), bool)
    for i in range(t):
        j = i
        while j >= 0:
            seen[i, j] = True
            up = j - 1 if parents is None else int(parents[j])
            j = up if up < j else -1
    return seen


def attention(c: Case):
    """(O, LSE, A) in float64: A = Σ p|v| bounds what rounding P can change."""
    q, kn, vn, k, v = (f64(x) for x in (c.q, c.k_new, c.v_new, c.k, c.v))
    table, cu = c.table.cpu(), c.cu.tolist()
    par = None if c.parents is None else c.parents.cpu().numpy()
    O = np.zeros((c.total, c.H, c.d))
    A = np.zeros_like(O)
    LSE = np.zeros((c.H, c.total))
    G = c.H // c.hkv
    for s, (n, t) in enumerate(zip(c.lens, c.new)):
        r = slice(cu[s], cu[s + 1])
        K = np.concatenate([rows_of(k, table, s, n).reshape(n, c.hkv, c.d), kn[r]])
        V = np.concatenate([rows_of(v, table, s, n).reshape(n, c.hkv, c.d), vn[r]])
        seen = np.concatenate([np.ones((t, n), bool), ancestors(None if par is None else par[r], t)], 1)
        for h in range(c.H):
            z = q[r, h] @ K[:, h // G].T * c.scale
            z[~seen] = -np.inf
            if t == 0:
                continue
            m = z.max(1, keepdims=True)
            e = np.exp(z - m)
            l = e.sum(1, keepdims=True)
            O[r, h] = (e / l) @ V[:, h // G]
            A[r, h] = (e / l) @ np.abs(V[:, h // G])
            LSE[h, r] = (m + np.log(l))[:, 0]
    return O, LSE, A


def score_bound(c: Case):
    """How far a score may be off after fp32 accumulation, from the sizes of q and k:
    (d + 8) roundings of partial sums of at most scale·|q||k|."""
    q, kn = np.abs(f64(c.q)), np.abs(np.nan_to_num(f64(c.k)))
    kn[kn > 1e4] = 0.0  # unused slots may hold anything
    big = 0.0
    if q.size:
        norm_k = np.sqrt((kn ** 2).sum(-1)).max() if kn.size else 0.0
        norm_k = max(norm_k, np.sqrt((f64(c.k_new) ** 2).sum(-1)).max())
        big = np.sqrt((q ** 2).sum(-1)).max() * norm_k * c.scale
    return (c.d + 8) * HALF_F32 * big + 2.0 ** -20


def weights(c: Case, lse, start=None):
    """weights_out in float64 at the slots in use (NaN elsewhere), from lse as given."""
    q, k = f64(c.q), f64(c.k)
    table, cu = c.table.cpu(), c.cu.tolist()
    lse = f64(lse)
    G = c.H // c.hkv
    out = np.full((c.n_pages, c.hkv, c.page), np.nan)
    for s, (n, t) in enumerate(zip(c.lens, c.new)):
        r = slice(cu[s], cu[s + 1])
        K = rows_of(k, table, s, n).reshape(n, c.hkv, c.d)
        seen = np.arange(n)[None] <= (n - t + np.arange(t))[:, None]
        for h in range(c.hkv):
            w = np.zeros(n)
            for g in range(h * G, (h + 1) * G):
                with np.errstate(over="ignore", invalid="ignore"):
                    p = np.exp(q[r, g] @ K[:, h].T * c.scale - lse[g, r][:, None])
                p[~seen] = 0.0
                p[~np.isfinite(lse[g, r])] = 0.0
                w += p.sum(0)
            for j in range(n):
                at = int(table[s, j // c.page]), h, j % c.page
                out[at] = w[j] + (0.0 if start is None else float(start[at]))
    return out


def selected(w, newest, budget):
    """kept of one (sequence, head) from its slots' weights and newness."""
    n = len(w)
    m = min(n, budget)
    key = np.where(np.isnan(w), -np.inf, w)
    # the newest first, all alike; then by weight; then by slot
    order = sorted(range(n), key=lambda j: (0, 0, 0, j) if newest[j] else (1, bool(np.isnan(w[j])), -key[j], j))
    order = order[:budget]
    stay = {j for j in order if j < m}
    move = iter(sorted(j for j in order if j >= m))
    return np.array([i if i in stay else next(move) for i in range(m)] + [-1] * (budget - m), np.int32)


def select(c: Case, budget, recent, seq_pos=None, by_position=True):
    w, pos, table = c.weights.cpu().numpy(), c.positions.cpu().numpy(), c.table.cpu()
    out = np.zeros((len(c.lens), c.hkv, budget), np.int32)
    for s, n in enumerate(c.lens):
        ws = rows_of(np.swapaxes(w, 1, 2), table, s, n).reshape(n, c.hkv)
        ps = rows_of(np.swapaxes(pos, 1, 2), table, s, n).reshape(n, c.hkv)
        for h in range(c.hkv):
            if by_position:
                newest = ps[:, h] >= int(seq_pos[s]) - recent
            else:
                newest = np.arange(n) >= n - recent
            out[s, h] = selected(ws[:, h], newest, budget)
    return out
