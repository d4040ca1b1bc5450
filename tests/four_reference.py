"""Plain 64-bit implementations of the 4-bit cache's format and of the page operators
for the tests.  They share nothing with the CUDA path."""
import math

import torch

import paged_reference

U = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def padded(D):
    return 64 if D <= 64 else 128 if D <= 128 else 256


def scales():
    """What the scale bytes 0 .. 226 stand for."""
    return torch.tensor([(e and 2.0 ** (e - 15) * (1 + m / 8)) or m * 2.0 ** -17
                         for e, m in ((b // 8, b % 8) for b in range(227))], dtype=torch.float64)


def nearest(x, values):
    """Index of the nearest of the ascending values, of two the even one."""
    at = torch.searchsorted(values, x).clamp(1, len(values) - 1)
    lo, hi = x - values[at - 1], values[at] - x
    up = (hi < lo) | ((hi == lo) & (at % 2 == 0))
    return torch.where(up, at, at - 1)


def scale_of(largest):
    return nearest(largest / 6, scales())


def to_four(x, scale=None):
    """Rows [..., P] in 64 bits -> (codes of the magnitudes [..., P], scale bytes [..., P / 16])."""
    g = x.unflatten(-1, (-1, 16))
    code = scale_of(g.abs().amax(-1)) if scale is None else scale
    s = scales()[code][..., None]
    u = torch.where(s > 0, g.abs() / s.clamp_min(2.0 ** -17), 0).clamp_max(6)
    return nearest(u, torch.tensor(U, dtype=torch.float64)).flatten(-2), code


def values(x, scale=None):
    """What rows stand for after they were put into 4 bits."""
    u, code = to_four(x, scale)
    v = torch.tensor(U, dtype=torch.float64)[u].unflatten(-1, (-1, 16)) * scales()[code][..., None]
    return v.flatten(-2) * torch.where(x < 0, -1.0, 1.0)


def pack(x):
    """Rows [..., P] -> bytes [..., P / 2], scale bytes [..., P / 16]."""
    u, code = to_four(x)
    c = (u | ((x < 0) & (u > 0)).long() << 3).to(torch.uint8)
    return c[..., 0::2] | c[..., 1::2] << 4, code.to(torch.uint8)


def unpack(data, scale):
    """Bytes -> what they stand for, [..., P]."""
    u = torch.tensor(U + [-x for x in U], dtype=torch.float64)
    c = torch.stack([data & 15, data >> 4], -1).flatten(-2).long()
    return (u[c].unflatten(-1, (-1, 16)) * scales()[scale.long()][..., None]).flatten(-2)


def check_rows(got_o, got_lse, ref, keys, dtype, D):
    """The row kernel's answer against paged_reference.attention()'s.

    Scores are off by e as in paged_reference.check_attention(), and so are the weights;
    as halves they are off by w = 2^-11 relative (fp16 outputs: two halves, 2^-22), or
    by 2^-37 of the row's largest.  The sum that O is divided by is of weights before
    they are rounded: |dO| <= (2 e + w) A + 2^-37 keys max |v|, and O is rounded once.
    """
    o, lse, a, size, vmax = ref
    u = paged_reference.HALF_STEP[dtype]
    w = 2.0 ** -22 if dtype == torch.float16 else 2.0 ** -11
    e = (D + 4) * 2.0 ** -24 * size + 2.0 ** -20
    tiny = 2.0 ** -37 * keys * vmax + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    bound = u * o.abs() + 1.01 * ((2 * e + w)[..., None] * a + tiny[..., None])
    got_o, empty = got_o.double().cpu(), torch.isneginf(lse)
    assert got_o.isfinite().all()
    assert (got_o[empty] == 0).all() and not torch.signbit(got_o[empty]).any()
    over = (got_o - o).abs() - bound
    assert (over <= 0).all(), f"O off by {(got_o - o).abs().max():.3e}, {over.max():.3e} over its bound"
    got_lse = got_lse.double().cpu()
    assert torch.equal(torch.isneginf(got_lse), empty)
    off = (got_lse[~empty] - lse[~empty]).abs()
    assert (off <= e[~empty] + 2.0 ** -22 * (1 + lse[~empty].abs())).all(), f"LSE off by {off.max():.3e}"


# ---------------------------------------------------------------------- pages
class Pages:
    """Tables, lengths and counts in Python lists, one step after another."""

    def __init__(self, table, seq_len, refs, page):
        self.table, self.seq_len, self.refs = table.tolist(), seq_len.tolist(), refs.tolist()
        self.page, self.width, self.N = page, table.shape[1], len(self.refs)

    def length(self, b):
        return max(0, min(self.seq_len[b], self.width * self.page))

    def have(self, n):
        return math.ceil(n / self.page)

    def free_list(self):
        return [p for p, n in enumerate(self.refs) if n <= 0]

    def grow(self, tokens):
        free, first, taken = self.free_list(), 0, []
        for b, t in enumerate(tokens):
            n = self.length(b)
            then = n + max(t, 0)
            need = self.have(then) - self.have(n) if then <= self.width * self.page else 0
            if then > self.width * self.page or (need and first + need > len(free)):
                taken.append(-2)
            else:
                for i in range(need):
                    p = free[first + i]
                    self.table[b][self.have(n) + i], self.refs[p] = p, 1
                if then > n:
                    self.seq_len[b] = then
                taken.append(need)
            first += need
        return taken

    def free(self, rows):
        for i, b in enumerate(rows):
            if not 0 <= b < len(self.table) or b in rows[:i]:
                continue
            for e in range(self.width):
                p = self.table[b][e]
                if e < self.have(self.length(b)) and 0 <= p < self.N and self.refs[p] > 0:
                    self.refs[p] -= 1
                self.table[b][e] = -1
            self.seq_len[b] = 0

    def fork(self, parent, child):
        B, free, taken, src = len(self.table), self.free_list(), [], []
        rank, was = 0, list(self.seq_len)
        for i, (x, y) in enumerate(zip(parent, child)):
            ok = 0 <= x < B and 0 <= y < B and y not in child[:i] and x not in child and was[y] <= 0
            n = self.length(x) if ok else 0
            tail = self.table[x][n // self.page] if ok and n % self.page else -1
            copied = 0 <= tail < self.N
            to = -1 if ok else -2
            if copied:
                to = free[rank] if rank < len(free) else -2
                rank += 1
            src.append(tail if copied and to >= 0 else -1)
            taken.append(to)
            if to == -2:
                continue
            row = [-1] * self.width
            for e in range(self.have(n)):
                p = row[e] = self.table[x][e]
                if to >= 0 and e == n // self.page:
                    row[e], self.refs[to] = to, 1
                elif 0 <= p < self.N:
                    self.refs[p] += 1
            self.table[y], self.seq_len[y] = row, n
        return src, taken

    def compact(self):
        live = [p for p, n in enumerate(self.refs) if n > 0]
        L = len(live)
        move = dict(zip([p for p in live if p >= L], [p for p in range(L) if self.refs[p] <= 0]))
        moved = [move.get(p, p if n > 0 else -1) for p, n in enumerate(self.refs)]
        for x, y in move.items():
            self.refs[y], self.refs[x] = self.refs[x], 0
        for b, row in enumerate(self.table):
            for e in range(self.have(self.length(b))):
                row[e] = move.get(row[e], row[e])
        return moved, move
