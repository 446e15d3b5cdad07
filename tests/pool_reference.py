"""Plain implementations of the calls on a cache's pages (python lists, one slot and page after another),
written from the definitions in include/sdcp.h; they share no code with the library."""

OK, LIMIT, BAD = 0, 2, 3


class Pool:
    def __init__(self, n_pages, page_tokens, n_slots, max_pages):
        self.n_pages, self.P, self.max_pages = n_pages, page_tokens, max_pages
        self.table = [[-1] * max_pages for _ in range(n_slots)]
        self.held = [0] * n_slots
        self.refs = [0] * n_pages

    def pages_of(self, tokens):
        return -(-tokens // self.P)

    def _inside(self, entries):
        return all(0 <= e < self.n_pages for e in entries)

    def fork(self, parent, length):
        before = list(self.held)
        status = []
        for b, a in enumerate(parent):
            if a == -1:
                status.append(OK)
            elif not 0 <= a < len(parent) or a == b or parent[a] != -1 or before[b] != 0 or not 0 <= before[a] <= self.max_pages or length[b] < 0:
                status.append(BAD)
            elif self.pages_of(length[b]) > before[a]:
                status.append(LIMIT)
            else:
                n = self.pages_of(length[b])
                if not self._inside(self.table[a][:n]):
                    status.append(BAD)
                    continue
                for i in range(n):
                    self.table[b][i] = self.table[a][i]
                    self.refs[self.table[a][i]] += 1
                self.held[b] = n
                status.append(OK)
        return status

    def reserve(self, kv_len, upto):
        free = [p for p in range(self.n_pages) if self.refs[p] == 0]
        begin = list(self.refs)
        status, copies, counted, dropped = [], [], 0, []
        for b, (n, u) in enumerate(zip(kv_len, upto)):
            if u <= n:
                status.append(OK)
                continue
            if n < 0 or not 0 <= self.held[b] <= self.max_pages or self.pages_of(n) > self.held[b]:
                status.append(BAD)
                continue
            end = self.pages_of(u)
            if end > self.max_pages:
                status.append(LIMIT)
                continue
            mine = range(n // self.P, min(self.held[b], end))
            if not self._inside([self.table[b][i] for i in mine]):
                status.append(BAD)
                continue
            want = [i for i in mine if begin[self.table[b][i]] > 1] + list(range(max(self.held[b], n // self.P), end))
            counted += len(want)
            if want and counted > len(free):
                status.append(LIMIT)
                continue
            for k, i in enumerate(want):
                page = free[counted - len(want) + k]
                old = self.table[b][i]
                if i < self.held[b]:
                    dropped.append(old)
                    if i == n // self.P and n % self.P:
                        copies.append((old, page, n % self.P, 0))
                self.table[b][i] = page
                self.refs[page] = 1
            self.held[b] = max(self.held[b], end)
            status.append(OK)
        for p in dropped:
            self.refs[p] -= 1
        return status, copies

    def release(self, keep):
        status = []
        for b, k in enumerate(keep):
            if k < 0:
                status.append(OK)
                continue
            h = self.held[b]
            if not 0 <= h <= self.max_pages:
                status.append(BAD)
                continue
            n = min(self.pages_of(k), h)
            if not self._inside(self.table[b][n:h]):
                status.append(BAD)
                continue
            for i in range(n, h):
                self.refs[self.table[b][i]] -= 1
                self.table[b][i] = -1
            self.held[b] = n
            status.append(OK)
        return status

    def compact(self, most):
        live = sum(r > 0 for r in self.refs)
        high = [p for p in reversed(range(live, self.n_pages)) if self.refs[p] > 0]
        holes = [p for p in range(live) if self.refs[p] <= 0]
        moves = list(zip(high, holes))[:most]
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        for b in range(len(self.held)):
            for i in range(min(self.held[b], self.max_pages)):
                self.table[b][i] = to.get(self.table[b][i], self.table[b][i])
        return live, [(a, b, self.P, 0) for a, b in moves]


def copy_pages(pages, copies, P, D):
    """pages: uint8 array [n_pages, heads, 2, bytes], changed in place; False if a record was left out."""
    good = True
    for a, b, tokens, _ in copies:
        if not (0 <= a < len(pages) and 0 <= b < len(pages) and a != b and 0 <= tokens <= P):
            good = False
            continue
        for g in range(D // 32):
            pages[b, :, :, g * P * 16:(g * P + tokens) * 16] = pages[a, :, :, g * P * 16:(g * P + tokens) * 16]
        at = P * D // 2
        pages[b, :, :, at:at + tokens * (D // 32)] = pages[a, :, :, at:at + tokens * (D // 32)]
    return good
