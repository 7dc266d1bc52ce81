"""Plain float64 attention and page bookkeeping that the attention tests compare
with, and the error bounds of the kernels' arithmetic."""
import numpy as np
import torch

U32 = 2.0 ** -23   # a whole fp32 step (tensor cores may truncate)
UB = 2.0 ** -8     # half a bf16 step


def attend(q, k, v, scale):
    """q [Hq, D]; k, v [n, Hkv, D] in float64.  Returns out, lse and their bounds.

    The bounds, term by term: a score is a sum of D products accumulated in
    fp32 and two more roundings (scale, subtraction): e_s.  The weights carry
    e_s twice (numerator and sum), the exponential's 2^-21 and the sum's n
    steps; they are rounded to bf16 once before they meet v (UB of sum w |v|)
    and the output once more (UB of |o|)."""
    Hq, D = q.shape
    n, Hkv = k.shape[:2]
    if n == 0:
        return (torch.zeros(Hq, D, dtype=torch.float64), torch.full((Hq,), -torch.inf, dtype=torch.float64),
                torch.zeros(Hq, D, dtype=torch.float64), torch.zeros(Hq, dtype=torch.float64))
    G = Hq // Hkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("hd,nhd->hn", q, kk) * scale
    m = s.amax(1, keepdim=True)
    e = torch.exp(s - m)
    tot = e.sum(1, keepdim=True)
    w = e / tot
    o = torch.einsum("hn,nhd->hd", w, vv)
    lse = (m + torch.log(tot)).squeeze(1)
    e_s = (D + 8) * U32 * scale * torch.einsum("hd,nhd->hn", q.abs(), kk.abs()).amax(1) + 4 * U32 * lse.abs()
    rel = 2 * e_s + 2.0 ** -20 + n * U32
    mass = torch.einsum("hn,nhd->hd", w, vv.abs())
    tol_o = (UB + rel)[:, None] * mass + UB * o.abs() + 1e-30
    return o, lse, tol_o, rel


def check(got, got_lse, want):
    o, lse, tol_o, tol_l = (torch.stack(x) for x in zip(*want))
    got, got_lse = got.double().cpu(), got_lse.double().cpu()
    assert torch.isfinite(got).all()
    assert ((got - o).abs() <= tol_o).all(), ((got - o).abs() - tol_o).max()
    empty = torch.isinf(lse)
    assert torch.equal(empty, torch.isinf(got_lse) & (got_lse < 0))
    assert ((got_lse - lse).abs()[~empty] <= tol_l[~empty]).all(), (got_lse - lse).abs()[~empty].max()


class Pages:
    """The page calls on plain lists: what tables, lens, refs and page contents have to be."""

    def __init__(self, n_pages, page, n_seqs, width):
        self.refs = [0] * n_pages
        self.rows = [[] for _ in range(n_seqs)]
        self.lens = [0] * n_seqs
        self.page, self.width = page, width
        self.data = {}   # (page, slot) -> token value

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r <= 0]

    def extend(self, seqs, counts):
        free, seen = self._free(), set()
        todo, asked = [], 0
        for s, c in zip(seqs, counts):
            if not 0 <= s < len(self.rows) or c < 0 or s in seen:
                continue
            seen.add(s)
            end = self.lens[s] + c
            if end > self.width * self.page:
                continue
            need = -(-end // self.page) - len(self.rows[s])
            if need and asked + need > len(free):
                asked += need
                continue
            if need:
                todo.append((s, free[asked:asked + need]))
            asked += need
            self.lens[s] = end
        for s, pages in todo:
            self.rows[s] += pages
            for p in pages:
                self.refs[p] = 1

    def write(self, seq, values):
        for i, x in enumerate(values):
            pos = self.lens[seq] - len(values) + i
            self.data[self.rows[seq][pos // self.page], pos % self.page] = x

    def read(self, seq):
        return [self.data[self.rows[seq][p // self.page], p % self.page] for p in range(self.lens[seq])]

    def fork(self, src, dst):
        free, n = self._free(), 0
        before = [(list(r), length) for r, length in zip(self.rows, self.lens)]
        seen = set()
        for a, b in zip(src, dst):
            if not (0 <= a < len(before) and 0 <= b < len(before)) or before[b][1] or b in seen:
                if 0 <= b < len(before):
                    seen.add(b)
                continue
            seen.add(b)
            row, length = before[a]
            full, part = divmod(length, self.page)
            if part:
                if n >= len(free):
                    n += 1
                    continue
                new = free[n]
                n += 1
                for i in range(part):
                    self.data[new, i] = self.data.get((row[full], i))
                self.refs[new] = 1
            for p in row[:full]:
                self.refs[p] += 1
            self.rows[b] = row[:full] + ([new] if part else [])
            self.lens[b] = length

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.rows):
                for p in self.rows[s]:
                    self.refs[p] -= 1
                self.rows[s], self.lens[s] = [], 0

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        holes = [p for p in self._free() if p < len(live)]
        for p, h in zip([p for p in live if p >= len(live)], holes):
            for i in range(self.page):
                if (p, i) in self.data:
                    self.data[h, i] = self.data[p, i]
            self.refs[h], self.refs[p] = self.refs[p], 0
            self.rows = [[h if x == p else x for x in r] for r in self.rows]

    def same_as(self, cache):
        tables = np.full((len(self.rows), self.width), -1)
        for i, r in enumerate(self.rows):
            tables[i, :len(r)] = r
        np.testing.assert_array_equal(cache.tables.cpu().numpy(), tables)
        np.testing.assert_array_equal(cache.lens.cpu().numpy(), self.lens)
        np.testing.assert_array_equal(cache.refs.cpu().numpy(), self.refs)
