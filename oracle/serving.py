"""Serving operators around the quantised cache (oracle; test infrastructure only).

Not on the source pages: attention of a batch over a shared quantised prefix and private
quantised tails, accumulated attention weights, eviction by them, and rotary positions.
Everything in float64 (angles in exact rational arithmetic), one token or pair at a time
where that keeps the definition in plain sight.

Pins (tests/test_serving.py): a batch of one with a prefix alone is ``attention.decode_attention``;
weights of one step sum to one per query head; eviction with equal masses keeps the lowest
tokens; a rotation followed by its inverse is the factor squared.
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from . import rrq
from .rrq import as_f64

# 2π to 60 digits, as a rational
TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def attention_shared(q, prefix, tails, lens, hkv, d, k_bits, v_bits, k_seed, v_seed, k_levels=None,
                     v_levels=None, scale=1.0):
    """q [B, hq, d]; prefix = (k_packed, k_norms, v_packed, v_norms) of T*hkv rows or None;
    tails = the same with B*cap*hkv rows or None; lens [B].  -> (out [B, hq, d],
    bound [B, hq] = Σ_t p_t ‖v̂_t‖), zeros for a sequence without tokens."""
    q = as_f64(q)
    batch, hq, _ = q.shape

    def decoded(part, bits, seed, levels, at):
        if part is None:
            return np.zeros((0, hkv, d))
        x = rrq.decode_exact(part[at], part[at + 1], bits, d, seed, levels)
        return x.reshape(-1, hkv, d)

    pk, pv = decoded(prefix, k_bits, k_seed, k_levels, 0), decoded(prefix, v_bits, v_seed, v_levels, 2)
    tk, tv = decoded(tails, k_bits, k_seed, k_levels, 0), decoded(tails, v_bits, v_seed, v_levels, 2)
    cap = tk.shape[0] // batch if batch else 0
    out, bound = np.zeros((batch, hq, d)), np.zeros((batch, hq))
    for b in range(batch):
        n = min(max(int(lens[b]), 0), cap) if cap else 0
        k = np.concatenate([pk, tk[b * cap:b * cap + n]])
        v = np.concatenate([pv, tv[b * cap:b * cap + n]])
        for h in range(hq):
            g = rrq.kv_group(h, hq, hkv)
            if k.shape[0] == 0:
                continue
            s = scale * (k[:, g] @ q[b, h])
            w = np.exp(s - s.max())
            p = w / w.sum()
            out[b, h] = p @ v[:, g]
            bound[b, h] = p @ np.linalg.norm(v[:, g], axis=1)
    return out, bound


def attention_mass(scores, hkv, mass=None, lens=None, decay=1.0):
    """scores [B, hq, T] -> (out [B, hkv, T], p [B, hq, T], distance to the head's largest
    score [B, hq, T], 0 where masked)."""
    s = np.asarray(scores, dtype=np.float64)
    batch, hq, t_len = s.shape
    out = np.zeros((batch, hkv, t_len)) if mass is None else as_f64(mass).copy()
    p, far = np.zeros_like(s), np.zeros_like(s)
    for b in range(batch):
        n = t_len if lens is None else min(max(int(lens[b]), 0), t_len)
        out[b, :, :n] *= decay
        for h in range(hq):
            row = s[b, h, :n]
            if n == 0 or np.all(row == -np.inf):
                continue
            x = row - row.max()
            w = np.exp(x)
            p[b, h, :n] = w / w.sum()
            far[b, h, :n] = np.where(np.isfinite(x), -x, 0.0)
            out[b, rrq.kv_group(h, hq, hkv), :n] += p[b, h, :n]
    return out, p, far


def evict(mass, lens, keep, sink, recent):
    """mass [B, hkv, cap] -> list over b of int arrays [hkv, m_b] of the kept tokens, ascending."""
    m = as_f64(mass)
    batch, hkv, cap = m.shape
    kept = []
    for b in range(batch):
        n = cap if lens is None else min(max(int(lens[b]), 0), cap)
        rows = []
        for g in range(hkv):
            if n <= keep:
                rows.append(np.arange(n))
                continue
            held = set(range(min(sink, n))) | set(range(n - recent, n))
            rest = [t for t in range(n) if t not in held]
            # NaN below −inf; −0 and +0 alike (Python compares them equal)
            rest.sort(key=lambda t: ((0, 0.0) if math.isnan(m[b, g, t]) else (-1, -m[b, g, t]), t))
            rows.append(np.array(sorted(list(held) + rest[:keep - len(held)])))
        kept.append(np.stack(rows) if rows else np.zeros((0, 0), int))
    return kept


def rope_frequencies(schedule, rot, base, stretch=1.0, original=8192.0, fast=32.0, slow=1.0):
    freqs = []
    if schedule == "ntk" and rot > 2:
        base = base * stretch ** (rot / (rot - 2))

    def pair_of(turns):
        return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

    for i in range(rot // 2):
        theta = base ** (-2 * i / rot)
        if schedule == "linear":
            theta = theta / stretch
        elif schedule == "yarn":
            lo, hi = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), rot - 1)
            ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            theta = theta * (1 - ramp) + theta / stretch * ramp
        freqs.append(theta)
    return np.array(freqs), (0.1 * math.log(stretch) + 1.0 if schedule == "yarn" else 1.0)


def angles(positions, freqs):
    """p·θ modulo one turn, in radians, from exact rationals: float64 [n, pairs]."""
    out = np.zeros((len(positions), len(freqs)))
    for i, f in enumerate(freqs):
        turn = Fraction(float(f)) / TWO_PI
        for k, p in enumerate(positions):
            t = int(p) * turn
            out[k, i] = float((t - math.floor(t)) * TWO_PI)
    return out


def rope(x, positions, freqs, interleaved=False, factor=1.0, inverse=False):
    """x [n, heads, d] -> (y float64, scale of the products |a| + |b| per coordinate)."""
    y = as_f64(x).copy()
    size = np.abs(y)
    phi = angles(positions, freqs) * (-1.0 if inverse else 1.0)
    half = len(freqs)
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = y[:, :, ia].copy(), y[:, :, ib].copy()
        c, s = factor * np.cos(phi[:, i])[:, None], factor * np.sin(phi[:, i])[:, None]
        y[:, :, ia], y[:, :, ib] = a * c - b * s, a * s + b * c
        size[:, :, ia] = size[:, :, ib] = abs(factor) * (np.abs(a) + np.abs(b))
    return y, size
