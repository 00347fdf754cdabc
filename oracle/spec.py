"""Oracle of the speculative decoding step over a paged cache, in 64 bits on the CPU.

Plain definitions, one request at a time: attention of drafted tokens, verification of
drafted tokens, the tree's visibility, and the pages' upkeep.
"""

import numpy as np


def ancestors(parents):
    """(n, n) truth values: row i sees itself and its ancestors.  A parent that is not a
    smaller index is none."""
    n = len(parents)
    m = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            m[i] = m[p]
        m[i, i] = True
    return m


def mask_words(seen, words):
    """Rows of truth values as 64-bit words (bits past the words are dropped)."""
    out = np.zeros((seen.shape[0], words), np.uint64)
    for i, j in zip(*np.nonzero(seen)):
        if j < 64 * words:
            out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


def attention(q, k, v, seen, scale):
    """q (T, Hq, D), k (S, Hkv, D), v (S, Hkv, Dv), seen (T, S): the result (T, Hq, Dv), the sums of
    weight times |v|, and per (token, head) the largest sum of |q k| and |score| of a key in
    sight.  Keys out of sight are left out before anything is computed with them."""
    T, hq, D = q.shape
    g = hq // k.shape[1]
    o, mag = np.zeros((T, hq, v.shape[2])), np.zeros((T, hq, v.shape[2]))
    prod, top = np.zeros((T, hq)), np.zeros((T, hq))
    for t in range(T):
        at = np.nonzero(seen[t])[0]
        if len(at) == 0:
            continue
        for h in range(hq):
            kk, vv = k[at, h // g], v[at, h // g]
            s = kk @ q[t, h] * scale
            prod[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * abs(scale)
            top[t, h] = np.abs(s).max()
            w = np.exp(s - s.max())
            w /= w.sum()
            o[t, h] = w @ vv
            mag[t, h] = w @ np.abs(vv)
    return o, mag, prod, top


def _weight(x):
    return np.where(np.isfinite(x) & (x > 0), x, 0.0)


def verify(tokens, parents, p, q, u, u_final, width):
    """One request: (path, next token).  p (and q, or None): (n, vocab) rows."""
    n = len(tokens)
    if n == 0:
        return [], -1
    V = p.shape[1]
    cur, path, first = 0, [0], 1
    while True:
        row = _weight(p[cur].astype(np.float64))
        draft = None if q is None else _weight(q[cur].astype(np.float64))
        w, mass, a, nxt = row.copy(), 1.0, 0.0, -1
        if len(path) < width:
            for i in range(first, n):
                if parents[i] != cur:
                    continue
                x = tokens[i]
                wx = w[x] if 0 <= x < V else 0.0
                qx = 1.0 if q is None else (draft[x] if 0 <= x < V else 0.0)
                if float(u[i]) * (mass * qx) < wx:
                    nxt = i
                    break
                if q is None:
                    mass -= wx
                    if 0 <= x < V:
                        w[x] = 0.0
                else:
                    a += mass
                    w = _weight(row - a * draft)
                    mass = float(w.sum())
        if nxt < 0:
            break
        cur, first = nxt, nxt + 1
        path.append(cur)
    if w.sum() <= 0:
        w = row
    if w.sum() <= 0:
        return path, -1
    cum = np.cumsum(w)
    v = int(np.searchsorted(cum, float(u_final) * cum[-1], side="right"))
    return path, min(v, int(np.nonzero(w > 0)[0].max()))


class Pool:
    """Page tables, counts and reference counts, followed one request at a time."""

    def __init__(self, table, counts, lens, refs, page_size):
        self.table, self.counts, self.lens, self.refs = (
            np.array(x, np.int64) for x in (table, counts, lens, refs))
        self.ps = page_size

    def _free(self):
        return list(np.nonzero(self.refs <= 0)[0])

    def resize(self, rows, new_lens, commit):
        refused, grow = 0, []
        for row, n in zip(rows, new_lens):
            need = -(-int(n) // self.ps)
            if not 0 <= row < len(self.counts) or n < 0 or need > self.table.shape[1]:
                refused += 1
                continue
            have = int(self.counts[row])
            for s in range(need, have):
                self.refs[self.table[row, s]] -= 1
            if need <= have:
                self.counts[row] = need
                if commit:
                    self.lens[row] = n
            else:
                grow.append((row, need, n))
        want = sum(need - int(self.counts[row]) for row, need, _ in grow)
        free = self._free()
        if want > len(free):
            return want - len(free), refused
        for row, need, n in grow:
            for s in range(int(self.counts[row]), need):
                self.table[row, s] = free.pop(0)
                self.refs[self.table[row, s]] = 1
            self.counts[row] = need
            if commit:
                self.lens[row] = n
        return 0, refused

    def fork(self, src, dst):
        """Status and the copies (from, to, tokens)."""
        ok, copies, refused = [], [], 0
        R = len(self.counts)
        for a, b in zip(src, dst):
            if not (0 <= a < R and 0 <= b < R) or a == b or self.counts[b] > 0 \
                    or -(-int(self.lens[a]) // self.ps) > self.counts[a]:
                refused += 1
            else:
                ok.append((a, b))
        want = sum(int(self.lens[a]) % self.ps > 0 for a, _ in ok)
        free = self._free()
        if want > len(free):
            return want - len(free), refused, []
        for a, b in ok:
            n = int(self.lens[a])
            full = n // self.ps
            self.table[b, :full] = self.table[a, :full]
            np.add.at(self.refs, self.table[a, :full], 1)
            if n % self.ps:
                self.table[b, full] = free.pop(0)
                self.refs[self.table[b, full]] = 1
                copies.append((int(self.table[a, full]), int(self.table[b, full]), n % self.ps))
            self.counts[b] = -(-n // self.ps)
            self.lens[b] = n
        return 0, refused, copies

    def place(self, row, pos):
        return int(self.table[row, pos // self.ps]), pos % self.ps
