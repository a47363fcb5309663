"""The paged cache's operators from their definitions, in 64 bits on the host, one
row at a time: what the tests of the cache and of the attention over it compare with."""
import numpy as np


def positions(q_start, kv_len):
    """(row, sequence, position) of every row that belongs to a sequence."""
    for s in range(len(kv_len)):
        for t in range(q_start[s], q_start[s + 1]):
            yield t, s, int(kv_len[s]) - int(q_start[s + 1] - t)


def visible(pos, length, window=0, first=None, prefix=None):
    lo, hi = 0, pos + 1
    if first is not None:
        lo = max(lo, int(first))
    if window > 0:
        lo = max(lo, pos - window + 1)
    if prefix is not None:
        hi = max(hi, int(prefix))
    return lo, min(hi, length)


def attention(q, k, v, table, q_start, kv_len, scale, cap=0.0, slopes=None, window=0, prefix=None, first=None):
    """q [T][Hq][D], k and v [pages][Hk][page][D] (as stored, any float type).  Returns out, lse, and for
    the tolerances: mean |v| under the weights, an upper bound of |score| terms, sum of weights over the largest,
    keys seen, largest |v| seen."""
    T, Hq, D = q.shape
    pages, Hk, ps, _ = k.shape
    g = Hq // Hk
    out = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    mean_abs, size = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    total, seen, top = np.ones((T, Hq)), np.zeros(T), np.zeros((T, Hq))
    q, mine = q.astype(np.float64), np.zeros(T, dtype=bool)
    for t, s, pos in positions(q_start, kv_len):
        mine[t] = True
        lo, hi = visible(pos, int(kv_len[s]), window, None if first is None else first[t],
                         None if prefix is None else prefix[s])
        j = np.arange(lo, max(lo, hi))
        page = table[s][j // ps] if len(j) else j
        ok = (page >= 0) & (page < pages)
        j, page = j[ok], page[ok]
        if not len(j):
            continue
        seen[t] = len(j)
        for h in range(Hq):
            kk = k[page, h // g, j % ps].astype(np.float64)
            vv = v[page, h // g, j % ps].astype(np.float64)
            with np.errstate(all="ignore"):
                x = kk @ q[t, h] * scale
                mag = np.abs(kk) @ np.abs(q[t, h]) * abs(scale)
                if cap:
                    x = cap * np.tanh(x / cap)
                if slopes is not None:
                    b = float(slopes[h]) * np.abs(pos - j)
                    x, mag = x - b, mag + np.abs(b)
                m = x.max()
                w = np.exp(x - m)
                out[t, h] = (w[:, None] * vv).sum(0) / w.sum()
                lse[t, h] = m + np.log(w.sum())
                mean_abs[t, h] = (w[:, None] * np.abs(vv)).sum(0) / w.sum()
                # the largest part of a score that carries weight
                size[t, h] = (mag * (w > 1e-12 * w.sum())).max()
                total[t, h], top[t, h] = w.sum(), np.abs(vv).max()
    return dict(out=out, lse=lse, mean_abs=mean_abs, size=size, total=total, seen=seen, top=top, mine=mine)


def attention_tolerance(r, f16):
    """Largest error the definition's roundings allow, element by element.
    Scores: products and sums of D <= 256 terms in 32 bits and up to eight more operations, each within 2^-24 of
    the terms' sum `size`; matrix cores and lane sums add in trees, so 2^-24 * 32 covers the sums of 256.
    Weights follow with that relative error (and 2^-22 of exp2 itself).  f16: each weight rounded (2^-11, or
    2^-25 / 64 where it is subnormal: weights are carried at 64 times their size) and the output rounded (2^-11, 2^-25)."""
    score = 2.0 ** -24 * 40 * (1 + r["size"])
    rel = 2 * score + 2.0 ** -20
    tol = rel[..., None] * r["mean_abs"]
    if f16:
        tol = tol + 2.0 ** -11 * r["mean_abs"] + 2.0 ** -11 * np.abs(r["out"]) + 2.0 ** -25
        tol = tol + (r["seen"][:, None] * 2.0 ** -31 * r["top"] / r["total"])[..., None]
    else:
        tol = tol + 2.0 ** -23 * np.abs(r["out"]) + 1e-37
    return tol, score + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0)))


def rope(x, pos, turns, pairs, magnitude=1.0):
    """x [T][H][D] turned by its rows' positions, in 64 bits."""
    x = x.astype(np.float64).copy()
    r = 2 * len(turns)
    a = 2 * np.pi * np.asarray(turns)[None, :] * np.asarray(pos, dtype=np.float64)[:, None]
    c, s = magnitude * np.cos(a)[:, None, :], magnitude * np.sin(a)[:, None, :]
    i0, i1 = (np.arange(0, r, 2), np.arange(1, r, 2)) if pairs else (np.arange(r // 2), np.arange(r // 2, r))
    x0, x1 = x[..., i0].copy(), x[..., i1].copy()
    x[..., i0], x[..., i1] = x0 * c - x1 * s, x1 * c + x0 * s
    return x


class Pages:
    """The pages' bookkeeping, one sequence at a time."""

    def __init__(self, refs, table, lens, page_size):
        self.refs, self.table, self.lens, self.ps = refs.copy(), table.copy(), lens.copy(), page_size

    def _row(self, s):
        return [int(p) for p in self.table[s] if 0 <= p < len(self.refs)]

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.lens):
                for p in self._row(s):
                    self.refs[p] -= 1
                self.table[s], self.lens[s] = -1, 0

    def fork(self, src, dst):
        n = len(self.lens)
        old_table, old_lens = self.table.copy(), self.lens.copy()
        pairs = [(a, b) for a, b in zip(src, dst) if 0 <= a < n and 0 <= b < n]
        for a, _ in pairs:
            for p in [int(x) for x in old_table[a] if 0 <= x < len(self.refs)]:
                self.refs[p] += 1
        for a, b in pairs:
            for p in [int(x) for x in old_table[b] if 0 <= x < len(self.refs)]:
                self.refs[p] -= 1
            self.table[b], self.lens[b] = old_table[a], old_lens[a]

    def extend(self, seqs, add):
        refs0 = self.refs.copy()
        free = [p for p in range(len(refs0)) if refs0[p] == 0]
        granted, copies, need_all, taken = [], [], 0, 0
        for s, a in zip(seqs, add):
            ok, need, copy, have, last = False, 0, False, 0, -1
            if 0 <= s < len(self.lens) and a >= 0:
                ln = int(self.lens[s])
                have, want = -(-ln // self.ps), -(-(ln + a) // self.ps)
                if want <= self.table.shape[1]:
                    last = int(self.table[s, have - 1]) if have else -1
                    copy = bool(a > 0 and ln % self.ps and 0 <= last < len(refs0) and refs0[last] > 1)
                    need = want - have + copy
                    ok = need_all + need <= len(free)
            need_all += need
            pair = (-1, -1)
            if ok:
                ids = free[taken:taken + need]
                taken += need
                begin = have - copy
                self.table[s, begin:begin + need] = ids
                for p in ids:
                    self.refs[p] = 1
                if copy:
                    self.refs[last] -= 1
                    pair = (last, ids[0])
                self.lens[s] = ln + a
            granted.append(int(ok))
            copies.append(pair)
        return np.array(granted, dtype=np.int32), np.array(copies, dtype=np.int32).reshape(-1, 2).T

    def compact(self):
        n = len(self.refs)
        live = [p for p in range(n) if self.refs[p] > 0]
        moved = np.full(n, -1, dtype=np.int32)
        moved[live] = live
        holes = [p for p in range(len(live)) if self.refs[p] <= 0]
        for a, b in zip([p for p in live if p >= len(live)], holes):
            moved[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        named = (self.table >= 0) & (self.table < n)
        self.table[named] = moved[self.table[named]]
        return moved
