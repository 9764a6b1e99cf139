"""fp64 CPU oracle of the paged cache: attention over pages, verification of drafted tokens, and the
upkeep of the pages.  TEST INFRASTRUCTURE ONLY, as the rest of this package; plain numpy loops, no
code shared with the product.

A cache is a pool k, v [n_pages, Hkv, 64, D] and a page table [B, max_pages]; token t of row b is slot
t % 64 of page table[b, t // 64].
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 64

BAD_INDEX, SIZE_MISMATCH, NO_PAGES, SHARED_PAGE, BAD_PROBS = 0x8, 0x4, 0x20, 0x40, 0x80


def rows(pool, table_row, L, h):
    """The first L entries of one row and KV head, [L, D] float64."""
    n = -(-L // PAGE)
    if n == 0:
        return np.zeros((0, pool.shape[3]))
    return np.concatenate([pool[p, h] for p in table_row[:n]])[:L].astype(np.float64)


def depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def visible(L, n, M, parent, window, sinks):
    """[M, L] bool: which entries each query sees (parent: a list, or None for the chain)."""
    parent = list(range(-1, M - 1)) if parent is None else list(parent)
    base, depth = L - n, depths(parent)
    see = np.zeros((M, L), dtype=bool)
    for m in range(min(n, M)):
        pos = base + depth[m]
        if base + m < 0:
            continue
        for t in range(max(0, min(base, L))):
            see[m, t] = window == 0 or pos - t < window or t < sinks
        a = m
        while a >= 0:
            at = base + depth[a]
            if base + a >= 0 and (window == 0 or pos - at < window or at < sinks):
                see[m, base + a] = True
            a = parent[a]
    return see


def attn(q, G, k, v, table, lens, parent=None, n_nodes=None, window=0, sinks=0, k_scale=1.0, v_scale=1.0):
    """(out [B, M, Hq, D], lse [B, M, Hq], mass [B, M, Hq, D] = sum p |v|, zabs [B, M, Hq] = the largest
    sum |q k| / sqrt(D) of a seen entry), float64."""
    B, M, Hq, D = q.shape
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    lse, zabs = np.full((B, M, Hq), -np.inf), np.zeros((B, M, Hq))
    q = q.astype(np.float64)
    for b in range(B):
        L = int(lens[b])
        n = M if n_nodes is None else int(n_nodes[b])
        see = visible(L, n, M, None if parent is None else parent[b], window, sinks)
        for h in range(Hq // G):
            kk, vv = rows(k, table[b], L, h) * k_scale, rows(v, table[b], L, h) * v_scale
            for m in range(M):
                s = see[m]
                if not s.any():
                    continue
                for g in range(h * G, h * G + G):
                    z = kk[s] @ q[b, m, g] / math.sqrt(D)
                    top = z.max()
                    e = np.exp(z - top)
                    lse[b, m, g] = top + math.log(e.sum())
                    p = e / e.sum()
                    out[b, m, g] = p @ vv[s]
                    mass[b, m, g] = p @ np.abs(vv[s])
                    zabs[b, m, g] = (np.abs(kk[s]) @ np.abs(q[b, m, g])).max() / math.sqrt(D)
    return out, lse, mass, zabs


def verify(p, q, tokens, parent, n_nodes, u_accept, u_sample):
    """(n_path [B], path [B, M], next [B], status): the walk as include/sgd.h states it."""
    B, M, V = p.shape
    n_path, path, nxt, status = np.zeros(B, np.int32), np.full((B, M), -1, np.int32), np.full(B, -1, np.int32), 0
    for b in range(B):
        n = M if n_nodes is None else int(n_nodes[b])
        if not 0 <= n <= M:
            status |= BAD_INDEX
            n = min(max(n, 0), M)
        if n == 0:
            continue
        par = [int(x) for x in parent[b][:n]]
        tok = [int(x) for x in tokens[b][:n]]
        usable = [True] * n
        if par[0] != -1:
            status |= BAD_INDEX
        for m in range(1, n):
            if not 0 <= tok[m] < V or not -1 <= par[m] < m:
                status |= BAD_INDEX
                usable[m] = False
        cur, walk = 0, [0]
        w, Z = p[b, 0].astype(np.float64), 1.0
        while True:
            for c in range(cur + 1, n):
                if not usable[c] or par[c] != cur:
                    continue
                qx = 1.0 if q is None else float(q[b, cur, tok[c]])
                if float(u_accept[b, c]) * qx * Z < w[tok[c]]:
                    cur = c
                    walk.append(c)
                    w, Z = p[b, c].astype(np.float64), 1.0
                    break
                if q is None:
                    r = w.copy()
                    r[tok[c]] = 0.0
                else:
                    r = np.maximum(w / Z - q[b, cur].astype(np.float64), 0.0)
                if r.sum() > 0:
                    w, Z = r, r.sum()
            else:
                break
        n_path[b] = len(walk)
        path[b, :len(walk)] = walk
        over = np.nonzero(np.cumsum(w) > float(u_sample[b]) * w.sum())[0]
        if len(over):
            nxt[b] = over[0]
        elif (w > 0).any():
            nxt[b] = np.nonzero(w > 0)[0][-1]
        else:
            nxt[b] = 0
            status |= BAD_PROBS
    return n_path, path, nxt, status


class Pages:
    """The state of a paged cache on the host, and the upkeep calls on it."""

    def __init__(self, k, v, table, lens, held, ref):
        self.k, self.v, self.table = k.copy(), v.copy(), table.copy()
        self.lens, self.held, self.ref = lens.copy(), held.copy(), ref.copy()

    def _free(self, n):
        pages = np.nonzero(self.ref == 0)[0]
        return pages[:n] if len(pages) >= n else None

    def reserve(self, add):
        """(new_lens, status)"""
        status = 0
        for b in range(len(add)):
            if (self.lens[b] < 0 or add[b] < 0 or not 0 <= self.held[b] <= self.table.shape[1] or
                    self.lens[b] > self.held[b] * PAGE or self.lens[b] + add[b] > self.table.shape[1] * PAGE):
                status |= SIZE_MISMATCH
            elif add[b]:  # the held pages that it would grow in
                last = min(int(self.held[b]), -(-(int(self.lens[b]) + int(add[b])) // PAGE))
                if (self.ref[self.table[b, self.lens[b] // PAGE:last]] > 1).any():
                    status |= SHARED_PAGE
        if status:
            return self.lens.copy(), status
        need = [max(0, -(-(int(L) + int(a)) // PAGE) - int(h)) for L, a, h in zip(self.lens, add, self.held)]
        pages = self._free(sum(need))
        if pages is None:
            return self.lens.copy(), NO_PAGES
        at = 0
        for b, n in enumerate(need):
            self.table[b, self.held[b]:self.held[b] + n] = pages[at:at + n]
            self.ref[pages[at:at + n]] = 1
            self.held[b] += n
            at += n
        return (self.lens + add).astype(np.int32), 0

    def append(self, k_new, v_new, cu):
        for b in range(len(self.lens)):
            n = int(cu[b + 1] - cu[b])
            for i in range(n):
                t = int(self.lens[b]) - n + i
                p = self.table[b, t // PAGE]
                self.k[p, :, t % PAGE] = k_new[:, cu[b] + i]
                self.v[p, :, t % PAGE] = v_new[:, cu[b] + i]

    def fork(self, src, dst):
        """status"""
        if len(set(dst.tolist())) < len(dst) or set(dst.tolist()) & set(src.tolist()) or (self.held[dst] != 0).any():
            return BAD_INDEX
        pages = self._free(int((self.lens[src] % PAGE != 0).sum()))
        if pages is None:
            return NO_PAGES
        at = 0
        for s, d in zip(src, dst):
            full = self.lens[s] // PAGE
            self.table[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                self.ref[p] += 1
            rest = self.lens[s] % PAGE
            if rest:
                new, old = pages[at], self.table[s, full]
                at += 1
                self.k[new, :, :rest], self.v[new, :, :rest] = self.k[old, :, :rest], self.v[old, :, :rest]
                self.table[d, full] = new
                self.ref[new] = 1
            self.held[d] = full + (rest > 0)
            self.lens[d] = self.lens[s]
        return 0

    def release(self, keep):
        for b in range(len(keep)):
            stay = -(-int(keep[b]) // PAGE)
            for p in self.table[b, stay:self.held[b]]:
                self.ref[p] -= 1
            self.held[b] = min(self.held[b], stay)

    def _compact(self, b, h, base, lst):
        src = [base + int(i) for i in lst]
        for x in (self.k, self.v):
            moved = [x[self.table[b, t // PAGE], h, t % PAGE].copy() for t in src]
            for i, row in enumerate(moved):
                t = base + i
                x[self.table[b, t // PAGE], h, t % PAGE] = row

    def accept(self, path, n_path, n_nodes):
        """new_lens"""
        new = self.lens - n_nodes + n_path
        for b in range(len(n_path)):
            for h in range(self.k.shape[1]):
                self._compact(b, h, int(self.lens[b] - n_nodes[b]), path[b, :n_path[b]])
        return new.astype(np.int32)

    def keep(self, idx, cu):
        """new_lens"""
        for b in range(len(self.lens)):
            for h in range(self.k.shape[1]):
                self._compact(b, h, 0, idx[h, cu[b]:cu[b + 1]])
        return (cu[1:] - cu[:-1]).astype(np.int32)
