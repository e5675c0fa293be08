"""The 8-bit paged key/value cache in numpy: its definition, token by token.

Append follows the library's definition in fp32, operation by operation, so
codes and scales can be compared bit for bit; read and attention are computed
in float64 from the codes.
"""

from __future__ import annotations

import numpy as np

BLOCK = 32


def value_position(i: int) -> int:
    """Where token i of a block lies in a row of the value codes."""
    j, t, e = i // 8, i % 8 // 2, i % 2
    return 8 * t + 2 * j + e


POSITIONS = np.array([value_position(i) for i in range(BLOCK)])


class Cache:
    """codes as the library lays them out; pages x heads x blocks."""

    def __init__(self, num_pages, H, D, page_size):
        n = page_size // BLOCK
        self.page_size, self.H, self.D = page_size, H, D
        self.k_codes = np.zeros((num_pages, H, n, D // 64, BLOCK, 64), np.int8)
        self.v_codes = np.zeros((num_pages, H, n, D, BLOCK), np.int8)
        self.k_scale = np.zeros((num_pages, H, n), np.float32)
        self.v_scale = np.zeros((num_pages, H, n), np.float32)

    def at(self, table_row, pos):
        return int(table_row[pos // self.page_size]), pos % self.page_size // BLOCK

    def block_codes(self, page, blk):
        """(k, v) codes of a block as [32, H, D]."""
        k = self.k_codes[page, :, blk].transpose(2, 0, 1, 3).reshape(BLOCK, self.H, self.D)
        v = self.v_codes[page, :, blk][:, :, POSITIONS].transpose(2, 0, 1)
        return k, v

    def set_block_codes(self, page, blk, k, v):
        self.k_codes[page, :, blk] = k.reshape(BLOCK, self.H, self.D // 64, 64).transpose(1, 2, 0, 3)
        self.v_codes[page, :, blk][:, :, POSITIONS] = v.transpose(1, 2, 0)

    def tokens(self, table_row, lo, hi):
        """(k, v) of tokens lo..hi-1 in float64, [hi - lo, H, D]."""
        ks, vs = np.zeros((2, max(0, hi - lo), self.H, self.D))
        pos = lo
        while pos < hi:
            page, blk = self.at(table_row, pos)
            i, n = pos % BLOCK, min(BLOCK - pos % BLOCK, hi - pos)
            k, v = self.block_codes(page, blk)
            ks[pos - lo:pos - lo + n] = k[i:i + n] * self.k_scale[page, :, blk, None].astype(np.float64)
            vs[pos - lo:pos - lo + n] = v[i:i + n] * self.v_scale[page, :, blk, None].astype(np.float64)
            pos += n
        return ks, vs


def requantize(x_new, codes_old, s_old):
    """One block and head: new tokens x_new [n, D] fp32, older codes [m, D] with scale
    s_old (m = 0: none). Returns (scale, older codes, new codes), fp32 arithmetic."""
    with np.errstate(all="ignore"):
        amax = np.max(np.abs(x_new)) if x_new.size else np.float32(0)
        s_old = np.float32(s_old) if len(codes_old) else np.float32(0)
        if not np.isfinite(amax) or np.isnan(s_old):
            return np.float32(np.nan), np.zeros_like(codes_old), np.zeros(x_new.shape, np.int8)
        s = max(s_old, np.float32(amax) / np.float32(127))
        if s == 0:
            return s, np.zeros_like(codes_old), np.zeros(x_new.shape, np.int8)
        new = np.clip(np.rint(x_new.astype(np.float32) / s), -127, 127).astype(np.int8)
        old = codes_old
        if len(codes_old) and s != s_old:
            old = np.rint(codes_old.astype(np.float32) * (s_old / s)).astype(np.int8)
        return s, old, new


def append(cache: Cache, k, v, table, starts, counts):
    """k, v: [B, T, H, D] float32 (BF16 values)."""
    for b in range(len(starts)):
        pos, end = int(starts[b]), int(starts[b]) + int(counts[b])
        while pos < end:
            first, stop = pos % BLOCK, min(BLOCK, end - (pos - pos % BLOCK))
            page, blk = cache.at(table[b], pos)
            codes = [c.copy() for c in cache.block_codes(page, blk)]
            t = pos - int(starts[b])
            for which, (x, scales) in enumerate(((k, cache.k_scale), (v, cache.v_scale))):
                for h in range(cache.H):
                    s, old, new = requantize(x[b, t:t + stop - first, h].astype(np.float32), codes[which][:first, h],
                                             scales[page, h, blk])
                    scales[page, h, blk] = s
                    codes[which][:first, h], codes[which][first:stop, h] = old, new
            cache.set_block_codes(page, blk, *codes)
            pos += stop - first


def attention_rows(q, k, v, sees, sm_scale):
    """q [R, D], k, v [L, D] float64; row r sees keys 0..sees[r]-1. Returns (o, lse, absolute
    weight sum p|v| / sum p) in float64: the last bounds what a relative error of p can do."""
    R, L = q.shape[0], k.shape[0]
    z = q.astype(np.float64) @ k.T * sm_scale
    hidden = np.arange(L)[None, :] >= np.asarray(sees)[:, None]
    z[hidden] = -np.inf
    m = np.max(z, 1, initial=-np.inf, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        p = np.where(hidden, 0.0, np.exp(z - np.where(np.isinf(m), 0.0, m)))
        l = p.sum(1, keepdims=True)
        o = np.where(l > 0, p @ v / l, 0.0)
        a = np.where(l > 0, p @ np.abs(v) / l, 0.0)
        lse = np.where(l > 0, m + np.log(l), -np.inf)[:, 0]
    return o, lse, a


def attention(cache: Cache, q, table, lengths, q_lengths, causal, sm_scale):
    """q [B, T, H, D] float32. Returns (o [B, T, H, D], lse [B, H, T], weight sums as o), float64; rows
    past q_lengths are 0 and -inf."""
    B, T, H, D = q.shape
    G = H // cache.H
    o, a = np.zeros((2, B, T, H, D))
    lse = np.full((B, H, T), -np.inf)
    for b in range(B):
        n, r = int(lengths[b]), int(q_lengths[b])
        k, v = cache.tokens(table[b], 0, n)
        sees = np.clip(n - r + 1 + np.arange(r), 0, n) if causal else np.full(r, n)
        for h in range(H):
            o[b, :r, h], lse[b, h, :r], a[b, :r, h] = attention_rows(q[b, :r, h], k[:, h // G], v[:, h // G], sees, sm_scale)
    return o, lse, a
