"""The attention-cache operators in numpy, 64 bits: rotation, the int8 block
rule, and attention with a causal mask, a sliding window and sinks (test
infrastructure only; shares no code with the HIP path).

Cache contents are kept here as plain [tokens, heads, d] arrays; `block_bytes`
alone knows the byte order of a cached block (include/kda.h), written as the
loop over elements that the header's index formula states.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def bf16(x):
    """Round to the nearest bf16 (ties to even); fp64 in and out."""
    f = np.asarray(x, np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    r = np.where(np.isnan(f), np.uint32(0x7FC00000), r)
    return r.view(np.float32).astype(np.float64)


def f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def rotate(x, pos, cos, sin, rot_dim, interleaved):
    """x [T, heads, d] at positions pos [T]; cos, sin [positions, rot_dim / 2] -> fp64."""
    y = np.array(x, np.float64)
    for i in range(rot_dim // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)
        c, s = cos[pos, i].astype(np.float64)[:, None], sin[pos, i].astype(np.float64)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


class Int8Blocks:
    """One request's cached keys (or values): codes and block scales, by the append rule."""

    def __init__(self, heads, d):
        self.codes = np.zeros((0, heads, d))
        self.scales = np.zeros((0, heads))

    def append(self, x, start):
        """x [T, heads, d] (the fp32 values) at positions start.. (fp32 quotients, as IEEE division gives them)."""
        x, heads, d = f32(x), x.shape[1], x.shape[2]
        end = start + len(x)
        nb = -(-end // BLOCK)
        codes, scales = np.zeros((nb * BLOCK, heads, d)), np.zeros((nb, heads))
        m = min(len(self.codes), nb * BLOCK)
        codes[:m] = self.codes[:m]
        scales[: min(len(self.scales), nb)] = self.scales[:nb]
        for b in range(start // BLOCK, nb):
            lo, hi = max(start, b * BLOCK), min(end, (b + 1) * BLOCK)
            old = scales[b] if lo > b * BLOCK else np.zeros(heads)
            new = np.maximum(old, f32(np.abs(x[lo - start: hi - start]).max(axis=(0, 2)) / 127.0))
            for h in range(heads):
                if new[h] > old[h] and lo > b * BLOCK:
                    c = codes[b * BLOCK: lo, h]
                    codes[b * BLOCK: lo, h] = np.clip(np.rint(f32(f32(c * old[h]) / new[h])), -127, 127)
                q = f32(x[lo - start: hi - start, h] / new[h]) if new[h] > 0 else np.zeros((hi - lo, d))
                codes[lo:hi, h] = np.clip(np.rint(q), -127, 127)
            scales[b] = new
        self.codes, self.scales = codes, scales

    def values(self, n):
        return self.codes[:n] * np.repeat(self.scales, BLOCK, axis=0)[:n, :, None]


def visible(p, n, window, sinks):
    """Which of the cached tokens 0..n-1 the query at position p sees."""
    j = np.arange(n)
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def attend(q, k, v, pos, scale, window=0, sinks=0):
    """q [T, Hq, d], k, v [n, H, d] (cached values), pos [T] -> (o, mag) [T, Hq, d] and the
    largest sum of |scale q k| terms over visible pairs [T, Hq]; mag is sum_j w_j |v_j|, what
    rounding errors of the weights are relative to."""
    T, hq, d = q.shape
    g = hq // k.shape[1]
    o, mag, load = np.zeros((T, hq, d)), np.zeros((T, hq, d)), np.zeros((T, hq))
    for t in range(T):
        see = visible(pos[t], len(k), window, sinks)
        for h in range(hq):
            kk, vv = k[see, h // g], v[see, h // g]
            x = scale * (kk @ q[t, h])
            w = np.exp(x - x.max())
            w /= w.sum()
            o[t, h] = w @ vv
            mag[t, h] = w @ np.abs(vv)
            load[t, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[t, h]))).max()
    return o, mag, load


def block_bytes(x, part, elem):
    """Bytes of one cached block part from x [32, d] (int8 codes, or bf16 values with elem 2)."""
    d = x.shape[1]
    out = np.zeros(32 * d, np.int8 if elem == 1 else np.uint16)
    e, g = 16 // elem, 2 // elem
    bits = x.astype(np.int8) if elem == 1 else (bf16(x).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    for t in range(32):
        for c in range(d):
            if part == 0:
                at = ((t // 16) * (d // e) + c // e) * 16 * e + (t % 16) * e + c % e
            else:
                slot = (t % 4) + 4 * (t // 16)
                at = (((c // (16 * g)) * 4 + (t % 16) // 4) * 16 + c % 16) * g * 8 + (c // 16 % g) * 8 + slot
            out[at] = bits[t, c]
    return out.view(np.uint8)
