"""A plain sequential model of the page operators (test infrastructure): the
pool as numpy arrays, each call one entry after the other."""
import numpy as np


class Pool:
    def __init__(self, rng, pages, ps, di, batch, max_pages):
        self.ps, self.pages = ps, pages
        row = [256, 32] + ([di] if di else [])
        self.data = [rng.integers(0, 256, (pages, ps, w)).astype(np.uint8) for w in row]
        self.table = np.full((batch, max_pages), -1, np.int32)
        self.seq_len = np.zeros(batch, np.int32)
        self.refs = np.zeros(pages, np.int32)
        self.refused = False

    def npages(self, n):
        return -(-int(n) // self.ps)

    def fill(self, rng, lens, shuffle=True):
        """Sequences of their own, on random free pages."""
        free = np.flatnonzero(self.refs == 0)
        if shuffle:
            free = rng.permutation(free)
        at = 0
        for b, n in enumerate(lens):
            c = self.npages(n)
            self.table[b, :c] = free[at:at + c]
            self.refs[free[at:at + c]] = 1
            self.seq_len[b] = n
            at += c

    def copy(self, src, dst):
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0 and a < self.pages and b < self.pages:
                for d in self.data:
                    d[b] = d[a]

    def _serve(self, wanted):
        """wanted: (pages, apply) of each valid entry, None for a refused one."""
        free = np.flatnonzero(self.refs == 0).tolist()
        at = 0
        out = []
        for w in wanted:
            if w is None or (w[0] > 0 and at + w[0] > len(free)):
                self.refused = True
                if w is not None:
                    at += w[0]
                out.append((-1, -1))
                continue
            out.append(w[1](free[at:at + w[0]]))
            at += w[0]
        return np.array(out, np.int32).reshape(-1, 2).T

    def _part(self, src, dst, rows):
        for d in self.data:
            d[dst, :rows] = d[src, :rows]

    def fork(self, parent, child, length=None):
        ps, room = self.ps, self.table.shape[1] * self.ps
        batch = len(self.seq_len)
        had = self.seq_len.copy()
        table = self.table.copy()
        seen, wanted = set(), []
        for i, (a, s) in enumerate(zip(parent, child)):
            ok = 0 <= s < batch and s not in seen
            if 0 <= s < batch:
                seen.add(int(s))
            ok = ok and 0 <= a < batch and a != s and had[s] == 0
            n = (min(had[a], length[i]) if length is not None else had[a]) if ok else -1
            if not ok or n < 0 or n > room:
                wanted.append(None)
                continue

            def apply(new, a=int(a), s=int(s), n=int(n)):
                whole = n // ps
                self.table[s] = -1
                self.table[s, :whole] = table[a, :whole]
                np.add.at(self.refs, table[a, :whole], 1)
                self.seq_len[s] = n
                if not new:
                    return -1, -1
                self.table[s, whole] = new[0]
                self.refs[new[0]] = 1
                self._part(table[a, whole], new[0], n % ps)
                return table[a, whole], new[0]

            wanted.append((int(n % ps != 0), apply))
        return self._serve(wanted)

    def resize(self, seq, new_len):
        ps, room = self.ps, self.table.shape[1] * self.ps
        refs = self.refs.copy()
        seen, wanted = set(), []
        for s, n in zip(seq, new_len):
            ok = 0 <= s < len(self.seq_len) and s not in seen
            if 0 <= s < len(self.seq_len):
                seen.add(int(s))
            if not ok or n < 0 or n > room:
                wanted.append(None)
                continue
            had = int(self.seq_len[s])
            cut = min(had, int(n))
            apart = cut % ps != 0 and refs[self.table[s, cut // ps]] > 1
            grown = max(0, self.npages(n) - self.npages(had))

            def apply(new, s=int(s), n=int(n), had=had, cut=cut, apart=apart):
                pair = (-1, -1)
                if apart:
                    old = self.table[s, cut // ps]
                    self._part(old, new[0], cut % ps)
                    self.refs[old] -= 1
                    self.refs[new[0]] = 1
                    self.table[s, cut // ps] = new[0]
                    pair = (old, new[0])
                    new = new[1:]
                a, b = self.npages(had), self.npages(n)
                for c in range(b, a):
                    self.refs[self.table[s, c]] -= 1
                    self.table[s, c] = -1
                for c in range(a, b):
                    self.table[s, c] = new[c - a]
                    self.refs[new[c - a]] = 1
                self.seq_len[s] = n
                return pair

            wanted.append((int(apart) + grown, apply))
        return self._serve(wanted)

    def compact(self):
        live = self.refs > 0
        n = int(live.sum())
        src = np.flatnonzero(live & (np.arange(self.pages) >= n))
        dst = np.flatnonzero(~live & (np.arange(self.pages) < n))
        to = np.arange(self.pages)
        to[src] = dst
        self.refs[dst], self.refs[src] = self.refs[src], 0
        for b in range(len(self.table)):
            c = self.npages(self.seq_len[b])
            self.table[b, :c] = to[self.table[b, :c]]
        self.copy(src, dst)
        moves = np.full((2, self.pages // 2), -1, np.int32)
        moves[0, :len(src)], moves[1, :len(dst)] = src, dst
        return moves, n
