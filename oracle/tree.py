"""Trees of drafted tokens in numpy, 64 bits: attention, the gated delta-rule
recurrence and the short convolution along a tree, the accepted path kept in an
int8 cache, and the upkeep of pages as plain loops (test infrastructure only;
shares no code with the HIP path).

A tree is a row of parents: -1 follows the last cached token, s < t follows node
s, below -1 there is no node; what does not descend from nodes before it is bad.
"""
from __future__ import annotations

import numpy as np

from . import attention as A


def ways(row):
    """Per entry: the nodes from its root to itself; [] for no node, None for a bad one."""
    out = []
    for t, p in enumerate(row):
        if p < -1:
            out.append([])
        elif p == -1:
            out.append([t])
        elif p < t and out[p]:
            out.append(out[p] + [t])
        else:
            out.append(None)
    return out


def attend(q, k, v, pos, row, scale, window=0, sinks=0):
    """q [T, Hq, d]; k, v [pos + T, H, d] (cached values, the tree's from slot pos on) -> as A.attend."""
    T, hq, d = q.shape
    o, mag, load = np.zeros((T, hq, d)), np.zeros((T, hq, d)), np.zeros((T, hq))
    for t, way in enumerate(ways(row)):
        if way is None:
            o[t] = np.nan
        elif way:
            at = np.concatenate([np.arange(pos), pos + np.asarray(way)])  # slots, in order of their positions
            n = len(at)
            o[t], mag[t], load[t] = (x[0] for x in A.attend(q[t: t + 1], k[at], v[at], [n - 1], scale, window, sinks))
    return o, mag, load


def commit(blocks, pos, path):
    """An A.Int8Blocks whose slots pos.. hold a tree: the path's rows to slots pos + i."""
    end = pos + len(path)
    src = list(range(end))
    for i, t in enumerate(path):
        src[pos + i] = pos + t
    if src == list(range(end)):
        return
    codes, scales = blocks.codes.copy(), blocks.scales.copy()
    for b in range(pos // A.BLOCK, -(-end // A.BLOCK)):
        mine = range(b * A.BLOCK, min(end, (b + 1) * A.BLOCK))
        new = np.max([blocks.scales[src[s] // A.BLOCK] for s in mine], axis=0)
        for s in mine:
            old, c = blocks.scales[src[s] // A.BLOCK], blocks.codes[src[s]]
            for h in range(len(new)):
                codes[s, h] = (c[h] if old[h] == new[h]
                               else np.clip(np.rint(A.f32(A.f32(c[h] * old[h]) / new[h])), -127, 127))
        scales[b] = new
    blocks.codes, blocks.scales = codes, scales


def recur(q, k, v, g, beta, row, S0):
    """One request: q, k, g, v [T, H, d], beta [T, H], S0 [H, d, d] -> o [T, H, d] and the states after each entry."""
    T, H, d = q.shape
    o, states = np.zeros((T, H, d)), [None] * T
    for t, way in enumerate(ways(row)):
        if way is None:
            o[t] = np.nan
            continue
        if not way:
            continue
        S = (S0 if len(way) == 1 else states[way[-2]]) * np.exp(np.maximum(g[t], -104.0))[..., None]
        u = v[t] - np.einsum("hkv,hk->hv", S, k[t])
        states[t] = S + (beta[t][:, None] * k[t])[..., None] * u[:, None]
        o[t] = np.einsum("hkv,hk->hv", states[t], q[t])
    return o, states


def recur_size(q, k, v, g, beta, row, S0):
    """What rounding errors of the closed form are relative to, [T, H, d]: its sums with every
    term's absolute value, |Qhat| |S0| + |Q| |(I + A)^-1| (I + |A| |(I + A)^-1|) (|V| + |Khat| |S0|)."""
    T, H, d = q.shape
    out = np.zeros((T, H, d))
    w = ways(row)
    for h in range(H):
        G = np.zeros((T, d))
        for t, way in enumerate(w):
            if way:
                G[t] = np.maximum(g[way, h], -104.0).sum(0)
        Am, Qm, Aa, Qa = (np.zeros((T, T)) for _ in range(4))
        for t, way in enumerate(w):
            for s in way or []:
                f = beta[s, h] * k[s, h] * np.exp(G[t] - G[s])
                Qm[t, s], Qa[t, s] = q[t, h] @ f, np.abs(q[t, h]) @ np.abs(f)
                if s != t:
                    Am[t, s], Aa[t, s] = k[t, h] @ f, np.abs(k[t, h]) @ np.abs(f)
        inv = np.abs(np.linalg.inv(np.eye(T) + Am))
        e = np.exp(G)
        rhs = np.abs(v[:, h]) + (np.abs(k[:, h]) * e) @ np.abs(S0[h])
        out[:, h] = (np.abs(q[:, h]) * e) @ np.abs(S0[h]) + Qa @ inv @ (np.eye(T) + Aa @ inv) @ rhs
    return out


def convolve(x, w, row, window):
    """x [T, C], w [C, W], window [W - 1, C] -> y [T, C] and the sums of |terms|."""
    W = w.shape[1]
    y, mag = np.zeros_like(x, np.float64), np.zeros_like(x, np.float64)
    for t, way in enumerate(ways(row)):
        if way is None:
            y[t] = np.nan
        elif way:
            rows = np.concatenate([window, x[way]])[-W:]
            y[t], mag[t] = (rows * w.T).sum(0), np.abs(rows * w.T).sum(0)
    return y, mag


class Pages:
    """Counts and tables, looked after by plain loops."""

    def __init__(self, refs, table, page_tokens):
        self.refs, self.table, self.pt = [int(x) for x in refs], [[int(x) for x in r] for r in table], page_tokens

    def free(self):
        return [p for p, n in enumerate(self.refs) if n <= 0]

    def release(self, first, last):
        for row, lo, hi in zip(self.table, first, last):
            for j, p in enumerate(row):
                if j * self.pt >= max(lo, 0) and (j + 1) * self.pt <= hi and p >= 0:
                    row[j] = -1
                    self.refs[p] -= 1

    def reserve(self, first, last):
        free, status = self.free(), []
        for row, lo, hi in zip(self.table, first, last):
            missing = 0
            for j, p in enumerate(row):
                if max(lo, 0) < hi and j * self.pt < hi and (j + 1) * self.pt > max(lo, 0) and p < 0:
                    if free:
                        row[j] = free.pop(0)
                        self.refs[row[j]] = 1
                    else:
                        missing += 1
            status.append(missing)
        return status

    def fork(self, src, dst, tokens):
        free, copies, status = self.free(), [], []
        for s, d, n in zip(src, dst, tokens):
            if n < 0:
                status.append(0)
                continue
            rows, width = len(self.table), len(self.table[0])
            if not (0 <= s < rows and 0 <= d < rows) or s == d or n > width * self.pt or any(p >= 0 for p in self.table[d]):
                status.append(2)
                continue
            whole, rest = divmod(n, self.pt)
            tail = self.table[s][whole] if rest else -1
            if tail >= 0 and not free:
                status.append(1)
                continue
            for j in range(whole):
                self.table[d][j] = self.table[s][j]
                if self.table[s][j] >= 0:
                    self.refs[self.table[s][j]] += 1
            if tail >= 0:
                p = free.pop(0)
                self.table[d][whole] = p
                self.refs[p] = 1
                copies.append((tail, p, rest))
            status.append(0)
        copies += [(-1, -1, 0)] * (len(src) - len(copies))
        return [list(x) for x in zip(*copies)], status

    def compact(self):
        held = [0] * len(self.refs)
        for row in self.table:
            for p in row:
                if p >= 0:
                    held[p] += 1
        movable = [p for p in range(len(held)) if self.refs[p] > 0 and held[p] == self.refs[p]][::-1]
        moves = [(s, d) for s, d in zip(movable, self.free()) if d < s]
        place = dict(moves)
        self.table = [[place.get(p, p) for p in row] for row in self.table]
        for s, d in moves:
            self.refs[d], self.refs[s] = self.refs[s], 0
        return moves


def closed_form(q, k, v, g, beta, row, S0, parts):
    """One request's o [T, H, d] by the closed form in the roundings that a kernel has: every
    product and sum in fp32, one after the other; parts: the operands in two bf16 parts, products
    of upper with lower ones, but not of two lower ones (0: in fp32; 1: without lower parts).
    exp(G_t - G_s) as the product of exp(G_t) and exp(-G_s) up to |G| of 60 (fp32: 16), past it
    pair by pair in fp32."""
    f, log2e = np.float32, np.float32(1.44269504)

    def split(x):
        if not parts:
            return [x]
        hi = A.bf16(x).astype(f)
        return [hi, A.bf16(x - hi).astype(f)] if parts == 2 else [hi]

    def dot(a, b):  # a [m, n], b [n, j] in parts
        s = np.zeros((a[0].shape[0], b[0].shape[1]), f)
        for x, y in [(a[0], b[0]), *[(x, b[0]) for x in a[1:]], *[(a[0], y) for y in b[1:]]]:
            for i in range(x.shape[1]):
                s = s + x[:, i: i + 1] * y[i: i + 1]
        return s

    T, H, d = q.shape
    o, w = np.zeros((T, H, d)), ways(row)
    on = np.array([[s in (x or ()) for s in range(T)] for x in w])
    for h in range(H):
        qh, kh, vh, gh, bh = (np.where(on.any(1).reshape(-1, *[1] * (x.ndim - 2)), x[:, h], 0).astype(f) for x in (q, k, v, g, beta))
        G = np.array([np.maximum(gh[x], f(-104)).sum(0, dtype=f) if x else np.zeros(d, f) for x in w])
        Kh, Qh = kh * np.exp2(G * log2e), qh * np.exp2(G * log2e)
        if np.abs(G).max() <= (60 if parts else 16):
            x = [y.T for y in split(bh[:, None] * kh * np.exp2(-G * log2e))]
            Am, Qm = dot(split(Kh), x), dot(split(Qh), x)
        else:
            Am, Qm = np.zeros((T, T), f), np.zeros((T, T), f)
            for s in range(T):
                x = kh[s] * np.exp2(np.where(on[:, s: s + 1], G - G[s], f(0)) * log2e)
                for to, y in ((Am, kh), (Qm, qh)):
                    to[:, s] = bh[s] * np.add.accumulate(y * x, axis=1, dtype=f)[:, -1]
        Am, Qm = np.where(on & ~np.eye(T, dtype=bool), Am, f(0)), np.where(on, Qm, f(0))
        W = Qm.copy()
        for j in range(T - 2, -1, -1):
            for i in range(j + 1, T):
                W[:, j] -= W[:, i] * Am[i, j]
        R = Qh - dot(split(W), split(Kh))
        o[:, h] = dot(split(R), split(S0[h].astype(f))) + dot(split(W), [vh])
    return o
