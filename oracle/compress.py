"""Plain fp64 definitions for compressed caches: the 4-bit pool, gathered
attention weight and eviction by it.  Numpy, one group, token or sequence at
a time; no code shared with the CUDA path.

16-bit values come and go as float64 arrays holding exactly representable
numbers; 4-bit pools are uint8 [NB, H, 9 * D] (the layout of
include/pagedattn.h).
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16


def round_bf16(x):
    """float64 -> nearest bfloat16 (ties to even), as float64."""
    f = np.asarray(x, dtype=np.float64).astype(np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(f), r, f).astype(np.float64)


def quantise(x):
    """x [..., D] float64 -> numbers n [..., D], scales and zero points [..., D/64]."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, 64)
    with np.errstate(invalid="ignore", over="ignore"):
        hi, lo, top = g.max(-1), g.min(-1), np.abs(g).max(-1)
        s = round_bf16(np.maximum((hi - lo) / 15.0, top / 2000.0))
    bad = ~np.isfinite(g).all(-1) | ~np.isfinite(s) | ((hi - lo) > np.finfo(np.float32).max)
    flat = (s == 0) | bad
    d = np.where(flat, 1.0, s)
    z = np.where(flat, 0.0, np.rint(-np.where(flat, 0.0, lo) / d)) + 0.0  # no negative zero
    n = np.clip(np.rint(np.where(flat[..., None], 0.0, g) / d[..., None]) + z[..., None], 0, 15)
    return n.reshape(x.shape).astype(np.uint8), np.where(bad, np.nan, s), z


def store_row(pool, block, head, row, x):
    """Quantise one token's row x [D] into (block, head, row) of a 4-bit pool."""
    D = x.shape[0]
    n, s, z = quantise(x)
    data = n[0::2] | n[1::2] << 4
    for c in range(D // 32):
        pool[block, head, c * 256 + row * 16:c * 256 + row * 16 + 16] = data[16 * c:16 * c + 16]
    for g in range(D // 64):
        zb = int(np.float16(z[g]).view(np.uint16))
        sb = 0x7FC0 if math.isnan(s[g]) else int(np.float32(s[g]).view(np.uint32) >> 16)
        word = 8 * D + (g * 16 + row) * 4
        pool[block, head, word:word + 4] = [zb & 255, zb >> 8, sb & 255, sb >> 8]


def parts(pool, D):
    """A 4-bit pool's numbers [NB, H, 16, D], scales and zero points [NB, H, 16, D/64]."""
    NB, H, _ = pool.shape
    n = np.zeros((NB, H, BLOCK, D))
    s = np.zeros((NB, H, BLOCK, D // 64))
    z = np.zeros((NB, H, BLOCK, D // 64))
    for t in range(BLOCK):
        for d in range(D):
            byte = pool[:, :, (d // 32) * 256 + t * 16 + (d % 32) // 2]
            n[:, :, t, d] = byte >> 4 if d % 2 else byte & 15
        for g in range(D // 64):
            w = pool[:, :, 8 * D + (g * 16 + t) * 4:][:, :, :4].astype(np.uint16)
            z[:, :, t, g] = (w[..., 0] | w[..., 1] << 8).astype(np.uint16).view(np.float16)
            s[:, :, t, g] = ((w[..., 2] | w[..., 3] << 8).astype(np.uint32) << 16).view(np.float32)
    return n, s, z


def values(pool, D):
    """What a 4-bit pool stands for, float64 [NB, H, 16, D]."""
    n, s, z = parts(pool, D)
    return np.repeat(s, 64, -1) * (n - np.repeat(z, 64, -1))


def attend(q, k, v, lens, tables, scale):
    """q [S, HQ, D]; k, v [NB, H, 16, D] float64.  Returns out [S, HQ, D], weights
    (a list of [HQ, L]) and sum_t w |v| [S, HQ, D]."""
    S, HQ, D = q.shape
    H = k.shape[1]
    G = HQ // H
    out, bound, weights = np.zeros((S, HQ, D)), np.zeros((S, HQ, D)), []
    for s in range(S):
        L = int(lens[s])
        w_all = np.zeros((HQ, L))
        for h in range(HQ if L else 0):
            rows_k = np.stack([k[tables[s, t // BLOCK], h // G, t % BLOCK] for t in range(L)])
            rows_v = np.stack([v[tables[s, t // BLOCK], h // G, t % BLOCK] for t in range(L)])
            x = scale * rows_k @ q[s, h]
            w = np.exp(x - x.max())
            w /= w.sum()
            w_all[h] = w
            out[s, h] = w @ rows_v
            bound[s, h] = w @ np.abs(rows_v)
        weights.append(w_all)
    return out, weights, bound


def gather_mass(mass_in, weights, decay):
    """decay * mass_in + the weights summed over heads; a copy, tails as they were."""
    out = np.array(mass_in, dtype=np.float64)
    for s, w in enumerate(weights):
        out[s, :w.shape[1]] = decay * out[s, :w.shape[1]] + w.sum(0)
    return out


def evict(mass, positions, history, L, keep, sinks, recent):
    """One sequence.  Returns (moves [(src, dst)], mass, positions, history) after it."""
    mass, positions = list(mass), list(positions)
    held, nxt = int(history[0]), int(history[1])
    if keep >= L:
        return [], mass, positions, (held, nxt)
    where = [positions[t] if t < held else nxt + t - held for t in range(L)]
    seen = nxt + L - held

    def rank(t):
        m = mass[t]
        if where[t] < sinks or where[t] >= seen - recent:
            return (0, 0.0, t)
        return (1, 0.0, t) if math.isnan(m) else (2, -m, t)

    stays = set(sorted(range(L), key=rank)[:keep])
    holes = [t for t in range(keep) if t not in stays]
    movers = [t for t in range(keep, L) if t in stays]
    moves = list(zip(movers, holes))
    for t in range(keep):
        positions[t] = where[t]
    for src, dst in moves:
        mass[dst], positions[dst] = mass[src], where[src]
    for t in range(keep, L):
        mass[t] = 0.0
    return moves, mass, positions, (keep, seen)
