"""Plain model (lists, no GPU) of cfz_kv8_free, _fork, _reserve and _compact, place by place from their
definitions."""


class Pages:
    def __init__(self, table, lengths, refs, page):
        self.table = [list(map(int, row)) for row in table]
        self.lengths, self.refs = list(map(int, lengths)), list(map(int, refs))
        self.page = page
        self.width = len(self.table[0])

    def named(self, page):
        return 0 <= page < len(self.refs)

    def held(self, row):
        return min(max(self.lengths[row], 0), self.width * self.page)

    def free(self, rows, keep=None):
        for i, row in enumerate(rows):
            if not 0 <= row < len(self.table):
                continue
            kept = max(0, keep[i]) if keep is not None else 0
            for e in range(-(-kept // self.page), self.width):
                if self.named(self.table[row][e]):
                    self.refs[self.table[row][e]] -= 1
                self.table[row][e] = -1
            self.lengths[row] = min(self.lengths[row], kept)

    def fork(self, parents, children):
        rows = range(len(self.table))
        done, pairs = set(), []
        for a, c in zip(parents, children):
            if a in rows and c in rows and c not in done and c not in parents:
                pairs.append((a, c))
            done.add(c)
        for a, c in pairs:
            n = self.held(a)
            for e in range(self.width):
                page = self.table[a][e] if e * self.page < n else -1
                page = page if self.named(page) else -1
                if page >= 0:
                    self.refs[page] += 1
                if self.named(self.table[c][e]):
                    self.refs[self.table[c][e]] -= 1
                self.table[c][e] = page
            self.lengths[c] = n

    def left_out(self, counts, max_new):
        """How many tokens of each row a reserve call has no place for."""
        return [max(0, n) - min(max(0, n), max_new, self.width * self.page - self.held(b))
                for b, n in enumerate(counts)]

    def reserve(self, counts, max_new):
        batch = len(self.table)
        source, target = [-1] * batch, [-1] * batch
        places = []
        for b in range(batch):
            n, held = min(max(counts[b], 0), max_new), self.held(b)
            last = min(self.width, -(-(held + n) // self.page)) if n else 0
            places += [(b, e) for e in range(held // self.page, last)]
        holders = {}
        for b, e in places:
            holders.setdefault(self.table[b][e], []).append((b, e))
        need = []
        for b, e in places:
            page = self.table[b][e]
            if not self.named(page):
                need.append((b, e))
            elif self.refs[page] > 1:
                mine = holders[page]
                if self.refs[page] > len(mine) or mine[0] != (b, e):
                    need.append((b, e))
        spare = [p for p, n in enumerate(self.refs) if n <= 0]
        if len(need) > len(spare):
            return source, target, len(need) - len(spare)
        for (b, e), page in zip(need, spare):
            old = self.table[b][e]
            self.table[b][e], self.refs[page] = page, 1
            if self.named(old):
                self.refs[old] -= 1
                if e * self.page < self.held(b):
                    source[b], target[b] = old, page
        return source, target, 0

    def compact(self):
        live = sum(n > 0 for n in self.refs)
        moves = []
        for low in range(live):
            if self.refs[low] <= 0:
                high = max(p for p, n in enumerate(self.refs) if n > 0)
                self.refs[low], self.refs[high] = self.refs[high], 0
                moves.append((high, low))
        to = dict(moves)
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return moves, live
