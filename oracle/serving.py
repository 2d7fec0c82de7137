"""Definitions of the serving operators in fp64 numpy: attention over packed prompts, and the 8-bit key/value
cache with its append, its attention and its eviction (the formulas of include/sda.h), one sequence and head at a
time, without blocking or reordering. Test infrastructure: no product code imports it.
"""
from __future__ import annotations

import numpy as np

from .fp8_quant import e4m3_decode as decode_e4m3, e4m3_encode


def encode_e4m3(x):
    """Codes of float32 values, NaN as 0x7f."""
    return np.where(np.isnan(x), np.uint8(0x7F), e4m3_encode(np.where(np.isnan(x), 0, x))).astype(np.uint8)


def attention_rows(q, k, v, visible, scale):
    """Rows of softmax(q k^T scale) v over the visible keys.

    q [n, d], k, v [m, d], visible [n, m]. Returns o [n, d], lse [n] (-inf where nothing is visible),
    p [n, m] and the spread sum_j p_j |v_j| that error bounds are stated in. Hidden keys do not enter,
    whatever they hold."""
    n, m = visible.shape
    o, spread = np.zeros((n, v.shape[1])), np.zeros((n, v.shape[1]))
    lse, p = np.full(n, -np.inf), np.zeros((n, m))
    for i in range(n):
        j = np.nonzero(visible[i])[0]
        if j.size == 0:
            continue
        s = (k[j] @ q[i]) * scale
        top = s.max()
        e = np.exp(s - top)
        lse[i] = top + np.log(e.sum())
        p[i, j] = e / e.sum()
        o[i] = p[i, j] @ v[j]
        spread[i] = p[i, j] @ np.abs(v[j])
    return o, lse, p, spread


def prompt_attention(q, k, v, seq_q, seq_k, causal=True, scale=None):
    """q [rows_q, H, d], k, v [rows_k, H_kv, d] -> o, lse, spread; rows outside the sequences are NaN."""
    H, d = q.shape[1:]
    g = H // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, spread = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    for s in range(len(seq_q) - 1):
        a, b, c, e = seq_q[s], seq_q[s + 1], seq_k[s], seq_k[s + 1]
        i, j = np.arange(b - a)[:, None], np.arange(e - c)[None]
        visible = j <= i + (e - c) - (b - a) if causal else np.ones((b - a, e - c), bool)
        for h in range(H):
            o[a:b, h], lse[a:b, h], _, spread[a:b, h] = attention_rows(q[a:b, h], k[c:e, h // g], v[c:e, h // g],
                                                                       visible, scale)
    return o, lse, spread


def wanted_scale(amax):
    """Smallest power of two s in [2^-126, 2^120] with amax <= 448 s."""
    e = -126
    while e < 120 and amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def recode(codes, ratio):
    """E4M3 codes of decode(codes) * ratio."""
    return encode_e4m3((decode_e4m3(codes) * ratio).astype(np.float32))


def append(k, v, seq, lens, table, block, pool, w=None):
    """Appends to `pool` (a dict of k_codes, v_codes, k_scale, v_scale arrays) and zeroes w, in place."""
    for b in range(len(lens)):
        n = seq[b + 1] - seq[b]
        for i in range(n):
            pos = lens[b] - n + i
            if pos // block != (pos - 1) // block or i == 0:      # first new token in this block
                stop = min(n, i + block - pos % block)
                blk = table[b, pos // block]
                for name, x in (("k", k), ("v", v)):
                    for h in range(x.shape[1]):
                        rows = x[seq[b] + i:seq[b] + stop, h]
                        mag = np.abs(rows[np.isfinite(rows)])
                        scale = wanted_scale(mag.max() if mag.size else 0.0)
                        old = pool[name + "_scale"][blk, h]
                        if pos % block:
                            scale = max(scale, float(old))
                            older = pool[name + "_codes"][blk, h, :pos % block]
                            pool[name + "_codes"][blk, h, :pos % block] = recode(older, np.float64(old) / scale)
                        pool[name + "_scale"][blk, h] = scale
                        # the quotient in fp32, as the kernel decides it
                        scaled = (rows.astype(np.float32) / np.float32(scale)).astype(np.float32)
                        pool[name + "_codes"][blk, h, pos % block:pos % block + stop - i] = encode_e4m3(scaled)
                if w is not None:
                    w[blk, :, pos % block:pos % block + stop - i] = 0


def cache_values(pool, name, table_row, length, block, h):
    """Values [length, d] of one sequence and key head."""
    t = np.arange(length)
    blk = table_row[t // block]
    return decode_e4m3(pool[name + "_codes"][blk, h, t % block]) * pool[name + "_scale"][blk, h].astype(np.float64)[:, None]


def cache_attention(q, seq, lens, table, block, pool, scale=None):
    """q [rows, H, d] -> o, spread and, per sequence, the weights [H_kv, len] summed over rows and heads."""
    H, d = q.shape[1:]
    H_kv = pool["k_scale"].shape[1]
    g = H // H_kv
    scale = d ** -0.5 if scale is None else scale
    o, spread, weights = np.full(q.shape, np.nan), np.full(q.shape, np.nan), []
    for b in range(len(lens)):
        a, e, t = seq[b], seq[b + 1], lens[b]
        pos = t - (e - a) + np.arange(e - a)
        visible = np.arange(t)[None] <= pos[:, None]
        wb = np.zeros((H_kv, t))
        for h in range(H):
            k, v = (cache_values(pool, n, table[b], t, block, h // g) for n in ("k", "v"))
            o[a:e, h], _, p, spread[a:e, h] = attention_rows(q[a:e, h], k, v, visible, scale)
            wb[h // g] += p.sum(0)
        weights.append(wb)
    return o, spread, weights


def kept_positions(w, length, keep, recent):
    """Positions that stay: the newest min(recent, n) and the heaviest older ones, ties to the lower, ascending."""
    n = min(length, keep)
    last = min(recent, n)
    older = sorted(range(length - last), key=lambda t: (0, 0.0, t) if np.isnan(w[t]) else (1, -w[t], t))  # NaN first, above infinity
    return np.array(sorted(older[:n - last]) + list(range(length - last, length)), np.int64)


def evict(lens, table, block, pool, w, dst_table, keep, recent):
    """Moves the kept tokens to dst_table's blocks in `pool` and w, in place; returns kept [B, H_kv, keep], dst_lens."""
    B, H_kv = len(lens), w.shape[1]
    kept, dst_lens = np.full((B, H_kv, keep), -1, np.int64), np.zeros(B, np.int64)
    for b in range(B):
        t = np.arange(lens[b])
        dst_lens[b] = min(lens[b], keep)
        for h in range(H_kv):
            stay = kept_positions(w[table[b, t // block], h, t % block], lens[b], keep, recent)
            kept[b, h, :len(stay)] = stay
            for first in range(0, len(stay), block):
                src = stay[first:first + block]
                blk, dst = table[b, src // block], dst_table[b, first // block]
                for name in ("k", "v"):
                    sc = pool[name + "_scale"][blk, h].astype(np.float64)
                    top = sc.max()
                    for i in range(len(src)):
                        pool[name + "_codes"][dst, h, i] = recode(pool[name + "_codes"][blk[i], h, src[i] % block],
                                                                  sc[i] / top)
                    pool[name + "_scale"][dst, h] = top
                w[dst, h, :len(src)] = w[blk, h, src % block]
    return kept, dst_lens
