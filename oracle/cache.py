"""Rotary positions, the paged cache and attention over it, in float64 on the CPU.

Written from the definitions alone, loop by loop over sequences, heads and tokens; shares no
code with the CUDA library. Rows are torch tensors; a cache is a dict of its arrays (the
layouts of lsh_cache in include/lsh_attn.h) that `append` changes in place.
"""
from __future__ import annotations

import math

import torch

SELF_LOGIT = -1.0e5
TINY = 2.0 ** -126  # smallest normal fp32: shorter keys count as zero, and the least scale


def rotate(row, angles, axis_dims, adjacent):
    """One row [d] (float64): pair p of all axes turned by angles[p]."""
    out = row.clone()
    at = p = 0
    for dims in axis_dims:
        for i in range(dims // 2):
            lo, hi = (at + 2 * i, at + 2 * i + 1) if adjacent else (at + i, at + dims // 2 + i)
            c, s = math.cos(angles[p]), math.sin(angles[p])
            out[lo] = row[lo] * c - row[hi] * s
            out[hi] = row[lo] * s + row[hi] * c
            p += 1
        at += dims
    return out


def angles_of(positions, freqs, axis_dims):
    """positions: one of each axis; freqs [pairs] fp32: the float64 angles of all pairs."""
    out, p = [], 0
    for a, dims in enumerate(axis_dims):
        for _ in range(dims // 2):
            out.append(int(positions[a]) * float(freqs[p]))
            p += 1
    return out


def rope(x, positions, freqs, axis_dims, adjacent=False, inverse=False):
    """x [B, H, n, d]; positions [axes, B, n] or [axes, n]. float64 result, not rounded."""
    B, H, n, _ = x.shape
    x = x.double()
    out = torch.empty_like(x)
    for b in range(B):
        for t in range(n):
            pos = positions[:, b, t] if positions.dim() == 3 else positions[:, t]
            ang = angles_of(pos, freqs, axis_dims)
            if inverse:
                ang = [-a for a in ang]
            for h in range(H):
                out[b, h, t] = rotate(x[b, h, t], ang, axis_dims, adjacent)
    return out


def empty(pages, heads, page_size, d, int8, fill=float("nan")):
    """A cache whose slots hold `fill` (int8: 99)."""
    dt = torch.int8 if int8 else torch.bfloat16
    f = 99 if int8 else fill
    c = {"k": torch.full((pages, heads, page_size, d), f, dtype=dt),
         "v": torch.full((pages, heads, page_size // 16, d, 16), f, dtype=dt),
         "key_inv_norm": torch.full((pages, heads, page_size), fill),
         "k_scale": None, "v_scale": None}
    if int8:
        c["k_scale"] = torch.full((pages, heads), fill)
        c["v_scale"] = torch.full((pages, heads), fill)
    return c


def scale_for(amax: float) -> float:
    """Smallest power of two s >= 2^-126 with amax <= 127 s."""
    s = TINY
    while 127 * s < amax:
        s *= 2
    return s


def _quant(x, s):
    q = torch.round(x / s).clamp(-127, 127)  # ties to even
    return torch.where(torch.isnan(x), torch.zeros_like(q), q)


def _v_row(cache, page, h, slot):
    return cache["v"][page, h, slot // 16, :, slot % 16]


def append(cache, rows, v, page_table, seq_len, n_valid=None, x=None):
    """Append bf16 rows [B, H, n, d] (rotated already) and v; the norms are those of `x`, the rows
    before the rotation (default: `rows`)."""
    B, H, n, _ = rows.shape
    P = cache["k"].shape[2]
    x = rows if x is None else x
    for b in range(B):
        nv = n if n_valid is None else int(n_valid[b])
        first = int(seq_len[b])
        for h in range(H):
            for t in range(nv):
                p = first + t
                page, slot = int(page_table[b, p // P]), p % P
                norm = float(x[b, h, t].double().norm())
                none = norm < TINY or (cache["k_scale"] is not None and math.isnan(norm))
                cache["key_inv_norm"][page, h, slot] = 0.0 if none else 1.0 / norm
                if cache["k_scale"] is None:
                    cache["k"][page, h, slot] = rows[b, h, t]
                    _v_row(cache, page, h, slot).copy_(v[b, h, t])
            if cache["k_scale"] is None:
                continue
            for pg in range(first // P, (first + nv - 1) // P + 1 if nv else 0):
                page = int(page_table[b, pg])
                lo, hi = max(first, pg * P), min(first + nv, (pg + 1) * P)
                old = max(0, first - pg * P)
                for name, new in (("k", rows), ("v", v)):
                    new = new[b, h, lo - first:hi - first].double()
                    fin = new[torch.isfinite(new)].abs()
                    was = float(cache[name + "_scale"][page, h]) if old else 0.0
                    s = max(was, scale_for(float(fin.max()) if fin.numel() else 0.0))
                    cache[name + "_scale"][page, h] = s

                    def put(slot, q):
                        if name == "k":
                            cache["k"][page, h, slot] = q.to(torch.int8)
                        else:
                            _v_row(cache, page, h, slot).copy_(q.to(torch.int8))
                    for slot in range(old if s != was else 0):
                        q = cache["k"][page, h, slot] if name == "k" else _v_row(cache, page, h, slot)
                        put(slot, torch.round(q.double() * (was / s)))
                    for i in range(hi - lo):
                        put(lo - pg * P + i, _quant(new[i], s))


def read(cache, page_table, b, h, count):
    """The first `count` cached tokens of sequence b: keys' rows, values, 1/||x||, in float64."""
    P = cache["k"].shape[2]
    p = torch.arange(count)
    page, slot = page_table[b].long()[p // P], p % P
    k = cache["k"][page, h, slot].double()
    v = cache["v"][page, h, slot // 16, :, slot % 16].double()
    if cache["k_scale"] is not None:
        k = k * cache["k_scale"][page, h].double()[:, None]
        v = v * cache["v_scale"][page, h].double()[:, None]
    return k, v, cache["key_inv_norm"][page, h, slot].double()


def attend(cache, x, page_table, seq_len, n_valid=None):
    """out, lse, and sum_j p_j |v_j| (the size of what is summed), in float64."""
    B, H, n, d = x.shape
    out = torch.zeros(B, H, n, d, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((B, H, n), -math.inf, dtype=torch.float64)
    for b in range(B):
        nv = n if n_valid is None else int(n_valid[b])
        if nv == 0:
            continue
        first = int(seq_len[b])
        for h in range(H):
            k, v, kinv = read(cache, page_table, b, h, first + nv)
            for t in range(nv):
                p = first + t
                l = (k[:p + 1] @ x[b, h, t].double()) * kinv[:p + 1] / math.sqrt(d)
                l[p] = SELF_LOGIT
                lse[b, h, t] = torch.logsumexp(l, 0)
                w = torch.softmax(l, 0)
                out[b, h, t] = w @ v[:p + 1]
                mag[b, h, t] = w @ v[:p + 1].abs()
    return out, lse, mag
