"""Plain form of the page and entry calls for the tests: lists on the host, one step at a time."""
import torch


class Pages:
    """The state of a pool as lists; each call as its description reads.  `flags`: whether a row was refused."""

    def __init__(self, page_size, refs, table, lens, held):
        self.P, self.refs, self.table = page_size, refs.tolist(), table.tolist()
        self.lens, self.held, self.flags = lens.tolist(), held.tolist(), False
        self.most = table.shape[1]

    def tensors(self):
        return [torch.tensor(v, dtype=torch.int32).reshape(shape) for v, shape in (
            (self.refs, (-1,)), (self.table, (len(self.lens), self.most)), (self.lens, (-1,)), (self.held, (-1,)))]

    def free(self, keep):
        for r, n in enumerate(keep):
            if n < 0:
                continue
            if not 0 <= self.held[r] <= self.most or n > self.held[r] * self.P:
                self.flags = True
                continue
            stay = -(-n // self.P)
            for i in range(stay, self.held[r]):
                p = self.table[r][i]
                self.table[r][i] = 0
                if 0 <= p < len(self.refs) and self.refs[p] > 0:
                    self.refs[p] -= 1
                else:
                    self.flags = True
            self.held[r], self.lens[r] = stay, n

    def _take(self, needs):
        """Pages for each row in order (None: refused), until the running sum passes the free ones."""
        free = [p for p, n in enumerate(self.refs) if n == 0]
        got, used = [], 0
        for n in needs:
            if n is None:
                got.append(None)
            elif n == 0:
                got.append([])
            else:
                got.append(free[used:used + n] if used + n <= len(free) else None)
                used += n
        for pages in got:
            for p in pages or []:
                self.refs[p] = 1
        return got

    def reserve(self, extra, width):
        needs = []
        for r, w in enumerate(extra):
            n, held = self.lens[r], self.held[r]
            if w < 0:
                needs.append(0)
                continue
            bad = n < 0 or not 0 <= held <= self.most or n + w > self.most * self.P
            if not bad and w > 0 and n % self.P and n // self.P < held:
                p = self.table[r][n // self.P]
                bad = not 0 <= p < len(self.refs) or self.refs[p] > 1
            self.flags |= bad
            needs.append(None if bad else max(0, -(-(n + w) // self.P) - held))
        slots, ok = [], []
        for r, pages in enumerate(self._take(needs)):
            ok.append(pages is not None)
            row = [-1] * width
            if pages is not None:
                for p in pages:
                    self.table[r][self.held[r]] = p
                    self.held[r] += 1
                for i in range(max(0, min(extra[r], width))):
                    j = self.lens[r] + i
                    row[i] = self.table[r][j // self.P] * self.P + j % self.P
            slots.append(row)
        return torch.tensor(slots, dtype=torch.int64).reshape(len(extra), width), torch.tensor(ok)

    def fork(self, parent):
        """ok, and the copies that are due: (from page, to page, places)."""
        needs = []
        for r, p in enumerate(parent):
            if p < 0:
                needs.append(0)
                continue
            bad = p >= len(self.lens) or self.held[r] != 0 or parent[p] >= 0
            bad = bad or self.lens[p] < 0 or not 0 <= self.held[p] <= self.most or self.lens[p] > self.held[p] * self.P
            self.flags |= bad
            needs.append(None if bad else int(self.lens[p] % self.P > 0))
        copies, ok = [], []
        for r, pages in enumerate(self._take(needs)):
            ok.append(pages is not None)
            if pages is None or parent[r] < 0:
                continue
            n = self.lens[parent[r]]
            full = n // self.P
            for i in range(full):
                p = self.table[parent[r]][i]
                self.table[r][i] = p
                self.refs[p] += 1
            if pages:
                self.table[r][full] = pages[0]
                copies.append((self.table[parent[r]][full], pages[0], n % self.P))
            self.lens[r], self.held[r] = n, full + len(pages)
        return torch.tensor(ok), copies


def compact(table, page, start, keep, count, places):
    """Moves (from slot, to slot) of ternary_kv_compact, and whether anything was refused."""
    moves, flags = [], False
    for b, (at, n) in enumerate(zip(start, count)):
        if at < 0 or n < 0 or n > len(keep[b]):
            flags = True
            n = 0 if at < 0 or n < 0 else len(keep[b])
        before = -1
        for i in range(n):
            k = keep[b][i]
            if k <= before or at + k >= places:
                flags = True
                break
            before = k
            moves.append((table[b][(at + k) // page] * page + (at + k) % page, table[b][(at + i) // page] * page + (at + i) % page))
    return moves, flags


def raw(cache):
    """A cache's four tensors as bytes and bit patterns, on the host."""
    return [t.view(torch.uint8).cpu() if t.element_size() == 1 else t.view(torch.int32).cpu()
            for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)]


def move(tensors, src, dst, page):
    """Slots moved in a cache's raw tensors, all read before any is written."""
    s, d = torch.tensor(src, dtype=torch.int64), torch.tensor(dst, dtype=torch.int64)
    for t in tensors:
        t[d // page, :, d % page] = t[s // page, :, s % page]
