"""The paged cache's operators in plain float64 loops, and small inputs for them (CPU tensors;
`to_cuda` moves a case to the device)."""
import math
from dataclasses import dataclass

import torch


@dataclass
class Cache:
    K: torch.Tensor
    V: torch.Tensor
    table: torch.Tensor
    lens: list
    page: int

    def rows(self, pages, s, g, slots):
        slots = torch.as_tensor(slots, dtype=torch.long)
        return pages[self.table[s].long()[slots // self.page], slots % self.page, g]


def make_cache(lens, h_kv, d, page, dtype, seed=0, spare=2, capacity=None, interleaved=False, stale=None):
    """Shuffled pages for sequences of `capacity` (default: lens) slots; -1 in unused table
    entries.  interleaved: K and V are slices of one [n_pages, 2, page, h_kv, d] tensor.  stale:
    the value of every row that no sequence holds."""
    g = torch.Generator().manual_seed(seed)
    cap = lens if capacity is None else capacity
    counts = [-(-c // page) for c in cap]
    n_pages = sum(counts) + spare
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(counts))), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(counts):
        table[s, :n] = order[at:at + n]
        at += n
    shape = (n_pages, 2, page, h_kv, d)
    both = torch.randn(shape, generator=g).to(dtype)
    if stale is not None:
        held = torch.zeros(n_pages, page, dtype=torch.bool)
        for s, L in enumerate(lens):
            j = torch.arange(L)
            held[table[s].long()[j // page], j % page] = True
        both = torch.where(held[:, None, :, None, None], both, torch.tensor(stale, dtype=dtype))
    K, V = both[:, 0], both[:, 1]
    if not interleaved:
        K, V = K.contiguous(), V.contiguous()
    return Cache(K, V, table, list(lens), page), both


def decode(c, Q, scale=None):
    """O, lse, the weights [nseq][h_kv][max_len] summed over each group, and error bounds:
    dx (of a score x_j, from float32 products and sums) and A = sum w |v|."""
    n, h_r, d = Q.shape
    h_kv = c.K.shape[2]
    G = h_r // h_kv
    scale = d ** -0.5 if scale is None else scale
    W = max(1, max(c.lens))
    O = torch.zeros(n, h_r, d, dtype=torch.float64)
    A = torch.zeros_like(O)
    lse = torch.full((n, h_r), -math.inf, dtype=torch.float64)
    dx = torch.zeros(n, h_r, dtype=torch.float64)
    xmax = torch.zeros(n, h_r, dtype=torch.float64)
    w = torch.zeros(n, h_kv, W, dtype=torch.float64)
    for s, L in enumerate(c.lens):
        if L == 0:
            continue
        for r in range(h_r):
            K = c.rows(c.K, s, r // G, range(L)).double()
            V = c.rows(c.V, s, r // G, range(L)).double()
            q = Q[s, r].double()
            x = (K @ q) * scale
            dx[s, r] = (d + 8) * 2.0 ** -23 * scale * (K.abs() @ q.abs()).max()
            xmax[s, r] = x.abs().max()
            lse[s, r] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[s, r]) if lse[s, r] > -math.inf else torch.zeros_like(x)
            O[s, r] = p @ V
            A[s, r] = p @ V.abs()
            w[s, r // G, :L] += p
    return O, lse, w, dx, A, xmax


def evict(c, score, pos, n_seen, budget, sink, window):
    """Moves rows of c.K, c.V in place; returns (score, pos, lens) with the tails cleared."""
    score, pos = score.clone(), pos.clone()
    lens = []
    for s, L in enumerate(c.lens):
        left = min(L, budget)
        lens.append(left)
        if L <= budget:
            continue
        for g in range(c.K.shape[2]):
            sc = score[s, g, :L].double().tolist()
            po = pos[s, g, :L].tolist()

            def order(j):
                safe = po[j] < sink or po[j] >= n_seen[s] - window
                v = sc[j]
                return (0, 0.0, j) if safe else (2, 0.0, j) if math.isnan(v) else (1, -v, j)

            kept = set(sorted(range(L), key=order)[:budget])
            dst = [j for j in range(budget) if j not in kept]
            src = [j for j in range(budget, L) if j in kept]
            for pages in (c.K, c.V):
                moved = c.rows(pages, s, g, src).clone()
                t = c.table[s].long()
                d = torch.tensor(dst, dtype=torch.long)
                pages[t[d // c.page], d % c.page, g] = moved
            score[s, g, dst] = score[s, g, src]
            pos[s, g, dst] = pos[s, g, src]
            score[s, g, left:L] = 0.0
            pos[s, g, left:L] = -1
    return score, pos, lens


def key_scores(values, row_ptr, col_idx, W, lens, base, B, h_kv):
    """score [nseq][h_kv][max(lens)] and the sum of the absolute terms."""
    G = W.shape[0] // h_kv
    Wd = W.double()
    width = max(1, max(lens))
    out = torch.zeros(len(lens), h_kv, width, dtype=torch.float64)
    mag = torch.zeros_like(out)
    for s, L in enumerate(lens):
        for qb in range(-(-L // B)):
            r = base[s] + qb
            for n in range(int(row_ptr[r]), int(row_ptr[r + 1])):
                kb = int(col_idx[n])
                i = qb * B + torch.arange(B)[:, None]
                j = kb * B + torch.arange(B)[None, :]
                live = (j <= i) & (i < L)
                A = torch.where(live, values[n].double(), 0.0)
                wide = min(B, L - kb * B)
                col = A.sum(1)[:, :wide]
                out[s, :, kb * B:kb * B + wide] += (Wd @ col).view(h_kv, G, wide).sum(1)
                mag[s, :, kb * B:kb * B + wide] += (Wd.abs() @ A.abs().sum(1)[:, :wide]).view(h_kv, G, wide).sum(1)
    return out, mag


def make_bsr(lens, B, h_s, dtype, seed=0, share=0.4, junk=None, gap=0):
    """Random kept blocks (the diagonal among them); junk fills the entries that must not count;
    gap leaves that many rows of no sequence between two sequences."""
    g = torch.Generator().manual_seed(seed)
    row_ptr, cols, vals, base = [0], [], [], []
    for L in lens:
        base.append(len(row_ptr) - 1)
        for qb in range(-(-L // B)):
            kept = [kb for kb in range(qb) if torch.rand(1, generator=g).item() < share] + [qb]
            for kb in kept:
                v = torch.rand(h_s, B, B, generator=g) / (B * len(kept))
                i = qb * B + torch.arange(B)[:, None]
                j = kb * B + torch.arange(B)[None, :]
                dead = (j > i) | (i >= L) | (j >= L)
                v = torch.where(dead, torch.tensor(0.0 if junk is None else junk), v)
                cols.append(kb)
                vals.append(v.to(dtype))
            row_ptr.append(len(cols))
        row_ptr.extend([len(cols)] * gap)
    values = torch.stack(vals) if vals else torch.zeros(0, h_s, B, B, dtype=dtype)
    return values, torch.tensor(row_ptr, dtype=torch.int32), torch.tensor(cols, dtype=torch.int32), base
