"""Page tables in plain Python, request after request: what kvq_extend_tables, kvq_fork_tables and kvq_trim_tables
leave behind."""


def up(a, b):
    return -(-a // b)


class Tables:
    """A pool and the rows of one table, as lists."""

    def __init__(self, num_pages, page_size, batch, max_pages):
        self.n, self.ps, self.maxp = num_pages, page_size, max_pages
        self.free = list(range(num_pages - 1, -1, -1))      # the list's memory
        self.count = num_pages
        self.refs, self.tags = [0] * num_pages, [0] * num_pages
        self.seq = [0] * batch
        self.rows = [[-1] * max_pages for _ in range(batch)]
        self.expected = [[0] * max_pages for _ in range(batch)]

    def take(self, place):
        page = self.free[place]
        self.refs[page] = 1
        self.tags[page] = (self.tags[page] + 1) % 2 ** 32
        return page

    def extend(self, offsets, total):
        """offsets: [batch + 1]; (slots with None where no request has a token, refused)."""
        slots, refused = [None] * total, []
        count, wanted = self.count, 0
        for r in range(len(self.seq)):
            old, off, n = self.seq[r], offsets[r], offsets[r + 1] - offsets[r]
            fits = old >= 0 and n >= 0 and off >= 0 and off + n <= total and old + n <= self.maxp * self.ps
            need = up(old + n, self.ps) - up(old, self.ps) if fits else 0
            wanted += need
            ok = fits and (need == 0 or wanted <= count)
            refused.append(0 if ok else 1)
            if ok:
                for i in range(need):
                    page = self.take(count - 1 - (wanted - need) - i)
                    self.rows[r][up(old, self.ps) + i] = page
                    self.expected[r][up(old, self.ps) + i] = self.tags[page]
                    self.count -= 1
                self.seq[r] = old + n
            if n > 0 and off >= 0 and off + n <= total:
                for t in range(n):
                    pos = old + t
                    slots[off + t] = self.rows[r][pos // self.ps] * self.ps + pos % self.ps if ok else -1
        return slots, refused

    def fork(self, parents, lens):
        before, count, wanted = list(self.seq), self.count, 0
        src, dst, refused = [], [], []
        for r, (p, n) in enumerate(zip(parents, lens)):
            fits = 0 <= p < len(before) and p != r and before[r] == 0 and 0 <= n <= before[p] <= self.maxp * self.ps
            part = fits and n % self.ps != 0
            wanted += part
            ok = fits and (not part or wanted <= count)
            refused.append(1 if p >= 0 and not ok else 0)
            pair = (-1, -1)
            if ok:
                whole = n // self.ps
                for i in range(whole):
                    page = self.rows[p][i]
                    self.rows[r][i], self.expected[r][i] = page, self.expected[p][i]
                    if 0 <= page < self.n:
                        self.refs[page] += 1
                if part:
                    page = self.take(count - wanted)
                    self.count -= 1
                    self.rows[r][whole], self.expected[r][whole] = page, self.tags[page]
                    pair = (self.rows[p][whole], page)
                self.seq[r] = n
            src.append(pair[0])
            dst.append(pair[1])
        return src, dst, refused

    def trim(self, keep):
        freed = set()
        for r, k in enumerate(keep):
            held = min(self.seq[r], self.maxp * self.ps)
            if not 0 <= k < held:
                continue
            for i in range(up(k, self.ps), up(held, self.ps)):
                page, self.rows[r][i] = self.rows[r][i], -1
                if 0 <= page < self.n and self.refs[page] > 0:
                    self.refs[page] -= 1
                    if self.refs[page] == 0:
                        freed.add(page)
            self.seq[r] = k
        for page in sorted(freed):
            self.free[self.count] = page
            self.count += 1
