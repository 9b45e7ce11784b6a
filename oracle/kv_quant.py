"""Oracle of the quantised KV cache (test infrastructure): NumPy float64, plain
loops. Written from the definition in include/s3r.h (s3r_paged_kvq); it shares
no code with the CUDA path.

A row x of one token and head: z = min x rounded down to bf16, s = bf16 of
float32 of (max x - z) / (2^bits - 1), n = (x - z) / s to the nearest whole
number (ties to even), clamped; it stands for s n + z.
"""
from __future__ import annotations

import numpy as np

TINY = 2.0 ** -100


def bf16_nearest(x):
    """float32 values -> bf16 bit patterns (uint16), ties to even (finite values)."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_down(x):
    """float32 values -> bf16 bit patterns, rounded towards minus infinity."""
    x = np.asarray(x, dtype=np.float32)
    u = x.view(np.uint32)
    up = (u >> 31).astype(bool) & ((u & 0xFFFF) != 0)          # negative and not a bf16 value: away from zero
    return ((u >> 16) + up).astype(np.uint16)


def bf16_value(bits):
    with np.errstate(invalid="ignore"):                        # NaN patterns
        return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise_rows(x, bits):
    """x [..., D] -> (n uint8 [..., D], s bits uint16 [...], z bits uint16 [...])."""
    x = np.asarray(x, dtype=np.float32)
    top = 2 ** bits - 1
    lead = x.shape[:-1]
    n = np.zeros(x.shape, dtype=np.uint8)
    s = np.full(lead, 0x3F80, dtype=np.uint16)
    z = np.zeros(lead, dtype=np.uint16)
    fine = np.isfinite(x).all(-1)
    z[~fine] = 0x7FC0
    if fine.any():
        r = x[fine].astype(np.float64)
        zb = bf16_down(x[fine].min(-1))
        zv = bf16_value(zb)
        sb = bf16_nearest(((r.max(-1) - zv) / top).astype(np.float32))
        sv = bf16_value(sb)
        flat = sv < TINY
        q = np.rint((r - zv[:, None]) / np.where(flat, 1.0, sv)[:, None])
        q = np.clip(q, 0, top)
        q[flat] = 0
        n[fine] = q.astype(np.uint8)
        s[fine] = np.where(flat, 0x3F80, sb)
        z[fine] = zb
    return n, s, z


def page_bytes(D, P, bits):
    return 2 * (P * D * bits // 8) + 8 * P


def _k_at(D, P, bits, t, d):
    """(byte, shift) of the key's number of token t, channel d."""
    byte = d * bits // 8
    return (byte // 16) * (P * 16) + t * 16 + byte % 16, (d * bits) % 8


def _v_at(D, P, bits, t, d):
    size = min(16, P * bits // 8)
    byte = t * bits // 8
    return P * D * bits // 8 + 4 * P + (byte // size) * (D * size) + d * size + byte % size, (t * bits) % 8


def write_row(page, D, P, bits, t, k_row, v_row):
    """Quantise one token's key and value rows into page (uint8 [page_bytes]), in place."""
    mask = 2 ** bits - 1
    half = P * D * bits // 8
    for row, at, par in ((k_row, _k_at, half), (v_row, _v_at, 2 * half + 4 * P)):
        n, s, z = quantise_rows(row, bits)
        for d in range(D):
            byte, shift = at(D, P, bits, t, d)
            page[byte] = (int(page[byte]) & ~(mask << shift) & 0xFF) | (int(n[d]) << shift)
        page[par + 4 * t:par + 4 * t + 4] = np.array([s, z], dtype="<u2").view(np.uint8)


def read_page(page, D, P, bits):
    """uint8 [page_bytes] -> (n_k [P, D], s_k [P], z_k [P], n_v, s_v, z_v), the parameters as float64."""
    mask = 2 ** bits - 1
    half = P * D * bits // 8
    t, d = np.meshgrid(np.arange(P), np.arange(D), indexing="ij")
    got = []
    for at, par in ((_k_at, half), (_v_at, 2 * half + 4 * P)):
        byte, shift = at(D, P, bits, t, d)
        w = page[par:par + 4 * P].copy().view("<u2").reshape(P, 2)
        got += [((page[byte].astype(np.int64) >> shift) & mask).astype(np.float64), bf16_value(w[:, 0]), bf16_value(w[:, 1])]
    return got


def append(pages, table, lens, k_new, v_new, bits, P, overwrite):
    """pages uint8 [N, H, page_bytes] and lens updated in place; k_new, v_new [S, n, H, D]."""
    S, n, H, D = k_new.shape
    for b in range(S):
        first = int(lens[b]) - overwrite
        for t in range(n):
            pos = first + t
            for h in range(H):
                write_row(pages[table[b, pos // P], h], D, P, bits, pos % P, k_new[b, t, h], v_new[b, t, h])
        lens[b] = first + n


def held_rows(pages, table_row, length, D, P, bits):
    """Keys and values [length, H, D] (float64) that a sequence's cache stands for, and their s, z [length, H]."""
    H = pages.shape[1]
    out = {x: [] for x in ("k", "v", "sk", "zk", "sv", "zv")}
    for i in range(-(-length // P)):
        heads = [read_page(pages[table_row[i], h], D, P, bits) for h in range(H)]
        for j, (x, sx, zx) in enumerate((("k", "sk", "zk"), ("v", "sv", "zv"))):
            n = np.stack([g[3 * j] for g in heads], 1)
            s = np.stack([g[3 * j + 1] for g in heads], 1)
            z = np.stack([g[3 * j + 2] for g in heads], 1)
            with np.errstate(invalid="ignore"):
                out[x].append(s[..., None] * n + z[..., None])
            out[sx].append(s)
            out[zx].append(z)
    return {x: np.concatenate(y)[:length] for x, y in out.items()}


def attend(q, held, scale, rows, positions_of_head=None):
    """One sequence: q [rows, Hq, D] over held rows; positions_of_head[h]: positions (with repeats) that head h's
    listed pages hold, None for all. Returns out, lse and, for error bounds, A = sum p |v| / sum p and
    B = sum p s_v / sum p per output."""
    R, Hq, D = q.shape
    L, H = held["sk"].shape
    G = Hq // H
    out, lse = np.zeros((R, Hq, D)), np.full((R, Hq), -np.inf)
    A, B = np.zeros((R, Hq, D)), np.zeros((R, Hq))
    for h in range(H):
        pos = np.arange(L) if positions_of_head is None else np.asarray(positions_of_head[h], dtype=np.int64)
        for r in range(R):
            seen = pos[pos <= L - R + r]
            if not len(seen):
                continue
            for g in range(G):
                x = held["k"][seen, h] @ q[r, h * G + g].astype(np.float64) * scale
                m = x.max()
                p = np.exp(x - m)
                tot = p.sum()
                p = p / tot
                out[r, h * G + g] = p @ held["v"][seen, h]
                lse[r, h * G + g] = m + np.log(tot)
                A[r, h * G + g] = p @ np.abs(held["v"][seen, h])
                B[r, h * G + g] = p @ held["sv"][seen, h]
    return out, lse, A, B
