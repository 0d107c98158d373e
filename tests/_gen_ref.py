"""Plain restatements that the tests of beams, cache slots and pages compare with:
64-bit torch for the choice of beams, Python lists for the pages of a cache."""
import math

import torch

F64 = torch.float64


def beam_tolerance(vocab: int) -> float:
    """What a value may be off by, beside its rounding to fp32: 2^-22 of a sum for an exponential, 2^-24 for each
    of ten additions and 2^-21 for the rescaling of each tile of 4096 that a thread adds (argument errors, |x| 2^-23,
    weigh at most 0.4 * 2^-23)."""
    return 2.0 ** -22 + 11 * 2.0 ** -24 + -(-vocab // 4096) * 2.0 ** -21


def beam_values(logits, scores, done=None, end=-1):
    """value(w, v) [batch, beams * vocab] in 64 bits, -inf where there is no candidate; and the beams that are refused."""
    batch, beams = scores.shape
    x = logits.to(F64).reshape(batch, beams, -1)
    V = x.shape[-1]
    ended = torch.zeros_like(scores, dtype=torch.bool) if done is None else done != 0
    bad_score = ~(scores <= 3.4028234663852886e38)            # NaN, +inf
    read = torch.isfinite(scores) & ~ended
    bad = bad_score | (read & ~(x.amax(-1) < math.inf))       # amax passes a NaN on
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    v = torch.where(torch.isfinite(x) & torch.isfinite(lse), x - lse, -math.inf)
    if end >= 0:
        only = torch.full((V,), -math.inf, dtype=F64, device=x.device)
        only[end] = 0.0
        v = torch.where(ended[..., None], only, v)
    v = v + torch.where(torch.isfinite(scores), scores.to(F64), -math.inf)[..., None]
    v = torch.where(bad[..., None], -math.inf, v)
    return v.reshape(batch, -1), bad


def beam_best(values, keep):
    """The keep largest of each row, equal ones by the lowest place (place -1: there is none)."""
    keep_here = min(keep, values.shape[1])
    s = torch.sort(values, dim=1, descending=True, stable=True)
    v, at = s.values[:, :keep_here], s.indices[:, :keep_here]
    at = torch.where(v > -math.inf, at, -1)
    if keep_here < keep:
        pad = keep - keep_here
        v = torch.cat([v, torch.full((v.shape[0], pad), -math.inf, dtype=F64, device=v.device)], 1)
        at = torch.cat([at, torch.full((v.shape[0], pad), -1, device=v.device)], 1)
    return v, at


class Pool:
    """A pool, its tables and the cache's pages as Python lists: contents[page] is any value."""

    def __init__(self, n_pages, page, rows, width, max_pos=1 << 20):
        self.n, self.page, self.width, self.max_pos = n_pages, page, width, max_pos
        self.table = [[-1] * width for _ in range(rows)]

    def refs(self):
        r = [0] * self.n
        for row in self.table:
            for p in row:
                if p >= 0:
                    r[p] += 1
        return r

    def free(self):
        return [p for p, r in enumerate(self.refs()) if r == 0]

    def grow(self, pos, new):
        """False: too few free pages; None: rows would go to a page that another place names, too."""
        want, refs = [], self.refs()
        for b, (p, n) in enumerate(zip(pos, new)):
            if n > 0 and p >= 0 and p + n <= min(self.max_pos, self.width * self.page):
                met = [(b, i) for i in range(p // self.page, (p + n - 1) // self.page + 1)]
                if any(self.table[b][i] >= 0 and refs[self.table[b][i]] > 1 for b, i in met):
                    return None
                want += [(b, i) for b, i in met if self.table[b][i] < 0]
        free = self.free()
        if len(want) > len(free):
            return False
        for (b, i), p in zip(want, free):
            self.table[b][i] = p
        return True

    def give(self, pos, window=0, sinks=0):
        for b, p in enumerate(pos):
            for i in range(self.width):
                first, last = i * self.page, (i + 1) * self.page - 1      # its positions
                kept = first < max(0, p)
                if window:
                    kept = kept and (first < sinks or last > p - window)
                if not kept:
                    self.table[b][i] = -1

    def fork(self, parent, pos):
        """(source, target, slots) of the copies, and the new positions; None: too few free pages."""
        free, refs, copies, rows, seen = self.free(), self.refs(), [], [], set()
        for i, p in enumerate(parent):
            if p < 0:
                rows.append([-1] * self.width)
                continue
            at, part = divmod(pos[p], self.page)
            first = p not in seen
            seen.add(p)
            row = list(self.table[p]) if first else self.table[p][:at] + [-1] * (self.width - at)
            if part and self.table[p][at] >= 0 and (not first or refs[self.table[p][at]] > 1):
                if len(copies) == len(free):
                    return None
                row[at] = free[len(copies)]
                copies.append((self.table[p][at], row[at], part))
            rows.append(row)
        self.table = rows
        return copies, [pos[p] if p >= 0 else 0 for p in parent]

    def compact(self, lo, hi):
        """{source: target}; None: too few free pages."""
        refs = self.refs()
        src = [p for p in range(lo, hi) if refs[p]]
        dst = [p for p in range(self.n) if not refs[p] and not lo <= p < hi]
        if len(dst) < len(src):
            return None
        to = dict(zip(src, dst))
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return to
