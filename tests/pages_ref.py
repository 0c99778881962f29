"""The page pool's calls from their definitions, one slot, row and page after the
other on the host; plain lists."""


class Pool:
    def __init__(self, n_pages, page_size, n_seq, max_pages):
        self.ps, self.most = page_size, max_pages * page_size
        self.refs = [0] * n_pages
        self.kv_len = [0] * n_seq
        self.table = [[-1] * max_pages for _ in range(n_seq)]
        self.moves, self.map = [], None
        self.bad = self.short = False

    def pages(self, n):
        return -(-n // self.ps)

    def _is_page(self, p):
        return 0 <= p < len(self.refs)

    def _fits(self, n):
        ok = 0 <= n <= self.most
        self.bad |= not ok
        return ok

    def reserve(self, tok_start):
        free = iter([p for p, r in enumerate(self.refs) if r == 0])
        self.moves = []
        for b, n in enumerate(self.kv_len):
            t0, t1 = tok_start[b], tok_start[b + 1]
            if not self._fits(n):
                continue
            if t0 < 0 or t1 < t0 or t1 - t0 > n:
                self.bad = True
                continue
            first = n - (t1 - t0)
            if first == n:
                continue
            for e in range(first // self.ps, (n - 1) // self.ps + 1):
                rows = max(0, first - e * self.ps)
                old = self.table[b][e] if rows else -1
                if rows:
                    if not self._is_page(old) or self.refs[old] <= 0:
                        self.bad, rows = True, 0
                    elif self.refs[old] == 1:
                        continue
                    else:
                        self.refs[old] -= 1
                new = next(free, -1)
                self.short |= new < 0
                self.table[b][e] = new
                if new >= 0:
                    self.refs[new] = 1
                if rows:
                    self.moves.append((old, new, rows))

    def fork(self, parent, child, length=None):
        had = list(self.kv_len)
        taken = set()
        for i, (p, c) in enumerate(zip(parent, child)):
            if p == -1 or c == -1:
                continue
            n_seq = len(had)
            if not (0 <= p < n_seq and 0 <= c < n_seq and p != c) or not self._fits(had[p]):
                self.bad = True
                continue
            m = had[p] if length is None else length[i]
            if not 0 <= m <= had[p] or had[c] != 0 or c in taken:
                self.bad = True
                continue
            taken.add(c)
            self.kv_len[c] = m
            for e in range(self.pages(m)):
                q = self.table[p][e]
                self.table[c][e] = q if self._is_page(q) else -1
                if self._is_page(q):
                    self.bad |= self.refs[q] <= 0
                    self.refs[q] += 1
                elif q != -1:
                    self.bad = True

    def _drop(self, b, e):
        p = self.table[b][e]
        if p == -1:
            return
        self.table[b][e] = -1
        if not self._is_page(p) or self.refs[p] <= 0:
            self.bad = True
        else:
            self.refs[p] -= 1

    def free(self, seq, keep=None):
        for i, b in enumerate(seq):
            k = 0 if keep is None else keep[i]
            if b == -1:
                continue
            if not 0 <= b < len(self.kv_len) or k < 0:
                self.bad = True
                continue
            old = self.kv_len[b]
            if not self._fits(old) or old <= k:
                continue
            self.kv_len[b] = k
            for e in range(self.pages(k), self.pages(old)):
                self._drop(b, e)

    def trim(self, window, sinks=0, tok_start=None):
        for b, n in enumerate(self.kv_len):
            if not self._fits(n):
                continue
            first = n
            if tok_start is not None:
                t0, t1 = tok_start[b], tok_start[b + 1]
                if t0 < 0 or t1 < t0 or t1 - t0 > n:
                    self.bad = True
                    continue
                first = n - (t1 - t0)
            for e in range(self.pages(n)):
                keys = range(e * self.ps, (e + 1) * self.ps)
                if all(j >= sinks and j <= first - window for j in (keys[0], keys[-1])):
                    self._drop(b, e)

    def compact(self):
        self.moves, self.map = [], [p if r else -1 for p, r in enumerate(self.refs)]
        lo, hi = 0, len(self.refs) - 1
        while lo < hi:
            if self.refs[lo]:
                lo += 1
            elif not self.refs[hi]:
                hi -= 1
            else:
                self.refs[lo], self.refs[hi] = self.refs[hi], 0
                self.map[hi] = lo
                self.moves.append((hi, lo, self.ps))
        if not self.moves:
            return
        for b, n in enumerate(self.kv_len):
            if not self._fits(n):
                continue
            for e in range(self.pages(n)):
                p = self.table[b][e]
                if p == -1:
                    continue
                if not self._is_page(p) or self.map[p] < 0:
                    self.bad = True
                else:
                    self.table[b][e] = self.map[p]
