"""Plain CPU oracle of the paged key-value cache: append, the attention of one
new token per sequence, eviction by accumulated weight.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path may import, call or
execute this module.  All arithmetic is float64, one sequence, head and slot
after the other; the E4M3 rows use the per-tensor quantiser of
``qkvp_oracle`` (pinned there) on one row at a time.

A cache is a dict of arrays: k [P, H, page, d_qk] and v [P, H, page, d_v]
(values, or uint8 codes with k_scale and v_scale [P, H, page]), pos and weight
[P, H, page], table [B, max_pages], lengths [B].
"""

from __future__ import annotations

import numpy as np

from .qkvp_oracle import dequantize, quantize


def _at(c, b, slot):
    page = c["k"].shape[2]
    return c["table"][b, slot // page], slot % page


def live_rows(c, b, h):
    """k, v (float64, de-quantised) of the live slots of sequence b, head h."""
    k, v = [], []
    for i in range(c["lengths"][b]):
        p, r = _at(c, b, i)
        if c.get("k_scale") is not None:
            k.append(dequantize(c["k"][p, h, r], c["k_scale"][p, h, r]))
            v.append(dequantize(c["v"][p, h, r], c["v_scale"][p, h, r]))
        else:
            k.append(c["k"][p, h, r].astype(np.float64))
            v.append(c["v"][p, h, r].astype(np.float64))
    d, dv = c["k"].shape[3], c["v"].shape[3]
    return np.array(k, np.float64).reshape(-1, d), np.array(v, np.float64).reshape(-1, dv)


def cache_append(c, k, v, pos, cu=None):
    """Stores k [H, T, d_qk], v [H, T, d_v] in place; returns the new lengths."""
    H, T, _ = k.shape
    B = len(c["lengths"])
    cu = np.arange(B + 1) if cu is None else cu
    lengths = np.array(c["lengths"])
    for b in range(B):
        for t in range(cu[b], cu[b + 1]):
            p, r = _at(c, b, lengths[b])
            for h in range(H):
                for name, row in (("k", k[h, t]), ("v", v[h, t])):
                    if c.get("k_scale") is not None:
                        c[name][p, h, r], c[name + "_scale"][p, h, r], _ = quantize(row)
                    else:
                        c[name][p, h, r] = row
                c["weight"][p, h, r] = 0.0
                c["pos"][p, h, r] = pos[t]
            lengths[b] += 1
    return lengths


def decode_attention(c, q, scale):
    """q [Hq, B, d_qk].  Returns a [B, Hq, d_v], lse [B, Hq], the probabilities
    p[b][hq] over the live slots, and for error bounds sum_i p_i |v_i| (like a)
    and max_i scale * sum_j |q_j k_ij| (like lse)."""
    Hq, B, _ = q.shape
    H, dv = c["k"].shape[1], c["v"].shape[3]
    a, absa = np.zeros((B, Hq, dv)), np.zeros((B, Hq, dv))
    lse, size = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    p = [[np.zeros(0)] * Hq for _ in range(B)]
    for b in range(B):
        for h in range(H if c["lengths"][b] else 0):
            k, v = live_rows(c, b, h)
            for hq in range(h * (Hq // H), (h + 1) * (Hq // H)):
                x = q[hq, b].astype(np.float64)
                s = scale * (k @ x)
                m = s.max()
                e = np.exp(s - m)
                p[b][hq] = e / e.sum()
                lse[b, hq] = m + np.log(e.sum())
                a[b, hq], absa[b, hq] = p[b][hq] @ v, p[b][hq] @ np.abs(v)
                size[b, hq] = np.max(abs(scale) * (np.abs(k) @ np.abs(x)))
    return a, lse, p, absa, size


def evict_slots(weight, pos, budget, recent):
    """The kept slots of one head in their new order, from the weights and
    positions of its live slots (more than ``budget``): new slot j holds what
    slot result[j] held."""
    newest = max(int(x) for x in pos)
    key = []
    for i, (w, x) in enumerate(zip(weight, pos)):
        w = float(w)
        protected = int(x) > newest - recent
        key.append((0 if protected else 1, 0.0 if protected else (np.inf if np.isnan(w) else -w),
                    0 if protected or not np.isnan(w) else 1, i))
    kept = sorted(k[3] for k in sorted(key)[:budget])
    movers = [i for i in kept if i >= budget]
    stays = set(i for i in kept if i < budget)
    return [j if j in stays else movers.pop(0) for j in range(budget)]


def cache_evict(c, budget, recent):
    """Evicts in place.  Returns slots [B, H, budget] and the new lengths."""
    B, H = len(c["lengths"]), c["k"].shape[1]
    slots = np.full((B, H, budget), -1, np.int32)
    names = [n for n in ("k", "v", "k_scale", "v_scale", "weight", "pos") if c.get(n) is not None]
    for b in range(B):
        n = c["lengths"][b]
        for h in range(H):
            if n <= budget:
                slots[b, h, :n] = np.arange(n)
                continue
            at = [_at(c, b, i) for i in range(n)]
            slots[b, h] = evict_slots([c["weight"][p, h, r] for p, r in at], [c["pos"][p, h, r] for p, r in at],
                                      budget, recent)
            for j, i in enumerate(slots[b, h]):
                if i != j:
                    for name in names:
                        c[name][at[j][0], h, at[j][1]] = c[name][at[i][0], h, at[i][1]]
    return slots, np.minimum(c["lengths"], budget)
