"""Causal attention over packed sequences with a window and sinks, and the split,
norm and rotation of a packed projection's rows, in float64, with gradients.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path may import, call or
execute this module.  Everything is written out per sequence and head from the
formulas."""

from __future__ import annotations

import numpy as np

D_V = 128


def seen(n: int, window, sinks: int) -> np.ndarray:
    """[n, n] bool: token i sees token j."""
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    ok = j <= i
    if window:
        ok &= (i - j < window) | (j < sinks)
    return ok


def spans(cu, T: int):
    """(start, end) of every sequence, offsets clamped into [0, T]."""
    if cu is None:
        return [(0, T)]
    c = np.clip(np.asarray(cu, np.int64), 0, T)
    return list(zip(c[:-1], c[1:]))


def attention(q, k, v, cu=None, window=None, sinks=0, scale=None, da=None):
    """q [Hq, T, d], k [H, T, d], v [H, T, 128] -> dict with a [T, Hq * 128], lse
    [Hq, T] and, with da [T, Hq * 128], dq, dk, dv; and the sums of absolute
    products that bound their errors: score [Hq, T] (the largest sum |q k| scale of
    a row's visible scores), pv [T, Hq * 128] (sum p |v|)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    Hq, T, d = q.shape
    H = k.shape[0]
    G = Hq // H
    scale = d ** -0.5 if scale is None else scale
    o = dict(a=np.zeros((T, Hq * D_V)), lse=np.full((Hq, T), -np.inf), score=np.zeros((Hq, T)), pv=np.zeros((T, Hq * D_V)))
    if da is not None:
        da = np.asarray(da, np.float64)
        o.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    for s, e in spans(cu, T):
        if e <= s:
            continue
        ok = seen(e - s, window, sinks)
        for h in range(Hq):
            c = slice(h * D_V, (h + 1) * D_V)
            qs, ks, vs = q[h, s:e], k[h // G, s:e], v[h // G, s:e]
            x = np.where(ok, scale * (qs @ ks.T), -np.inf)
            m = x.max(-1, keepdims=True)
            w = np.exp(x - m)
            p = w / w.sum(-1, keepdims=True)
            o["lse"][h, s:e] = (m + np.log(w.sum(-1, keepdims=True)))[:, 0]
            o["a"][s:e, c] = p @ vs
            o["pv"][s:e, c] = p @ np.abs(vs)
            o["score"][h, s:e] = np.where(ok, scale * (np.abs(qs) @ np.abs(ks).T), 0).max(-1)
            if da is None:
                continue
            g = da[s:e, c]
            dp = g @ vs.T
            ds = p * (dp - (p * dp).sum(-1, keepdims=True))
            o["dq"][h, s:e] = scale * (ds @ ks)
            o["dk"][h // G, s:e] += scale * (ds.T @ qs)
            o["dv"][h // G, s:e] += p.T @ g
    return o


def gradient_bounds(q, k, v, da, cu=None, window=None, sinks=0, scale=None):
    """How far dq, dk and dv may be off, from the arithmetic alone: float32 sums of
    exact products, probabilities and ds each rounded to bf16 for the products that
    they enter, da . a formed with the bf16 a, and the results rounded to bf16.

    half = 2^-8 (half a bf16 step), u = 2^-23 (a float32 step that may truncate).
      scores      es = (d + 8) u scale sum |q k|
      p           ep = 2 es + 2^-19 (1 + |lse|), relative
      dp          ed = 136 u sum |da v|
      da . a      ea = sum |da| ((half + ep) sum p |v| + half |a|) + 136 u sum |da a|
      ds          half |ds| + ep |ds| + p (ed + ea)
    """
    q, k, v, da = (np.asarray(x, np.float64) for x in (q, k, v, da))
    Hq, T, d = q.shape
    G = Hq // k.shape[0]
    scale = d ** -0.5 if scale is None else scale
    half, u = 2.0 ** -8, 2.0 ** -23
    f = attention(q, k, v, cu, window, sinks, scale, da)
    b = dict(dq=half * np.abs(f["dq"]), dk=half * np.abs(f["dk"]), dv=half * np.abs(f["dv"]))
    for s, e in spans(cu, T):
        if e <= s:
            continue
        ok = seen(e - s, window, sinks)
        for h in range(Hq):
            c = slice(h * D_V, (h + 1) * D_V)
            qs, ks, vs, g, lse = q[h, s:e], k[h // G, s:e], v[h // G, s:e], da[s:e, c], f["lse"][h, s:e, None]
            p = np.where(ok, np.exp(scale * (qs @ ks.T) - lse), 0)
            es = (d + 8) * u * scale * (np.abs(qs) @ np.abs(ks).T).max(-1, keepdims=True)
            ep = 2 * es + 2.0 ** -19 * (1 + np.abs(lse))
            dp = g @ vs.T
            ds = p * (dp - (p * dp).sum(-1, keepdims=True))
            a = p @ vs
            ed = 136 * u * (np.abs(g) @ np.abs(vs).T)
            ea = ((np.abs(g) * ((half + ep) * (p @ np.abs(vs)) + half * np.abs(a))).sum(-1, keepdims=True)
                  + 136 * u * (np.abs(g) * np.abs(a)).sum(-1, keepdims=True))
            ead = p * (ed + ea)
            np.einsum("ii->i", ead)[ok.sum(-1) == 1] = 0      # a token alone passes on exactly nothing
            es_ = (half + ep) * np.abs(ds) + ead
            long = (e - s) * u     # the sums' own rounding
            b["dq"][h, s:e] += scale * (es_ @ np.abs(ks)) + long * scale * (np.abs(ds) @ np.abs(ks))
            b["dk"][h // G, s:e] += scale * (es_.T @ np.abs(qs)) + G * long * scale * (np.abs(ds).T @ np.abs(qs))
            b["dv"][h // G, s:e] += ((half + ep) * p).T @ np.abs(g) + G * long * (p.T @ np.abs(g))
    return f, b


# ---------------------------------------------------------------------------
# Split, norm, rotation
# ---------------------------------------------------------------------------

def angles(pos, d: int, base: float = 10000.0, sections=None) -> np.ndarray:
    """[T, d / 2] angles; pos [T], or [axes, T] with sections."""
    w = base ** (-2.0 * np.arange(d // 2) / d)
    pos = np.atleast_2d(np.asarray(pos, np.float64))
    axis = np.zeros(d // 2, int) if sections is None else np.repeat(np.arange(len(sections)), sections)
    return pos[axis].T * w


def rotate(x, ang, back=False):
    """Pairs (i, i + d / 2) of x [T, d] turned by ang [T, d / 2]."""
    h = x.shape[-1] // 2
    c, s = np.cos(ang), -np.sin(ang) if back else np.sin(ang)
    return np.concatenate([x[:, :h] * c - x[:, h:] * s, x[:, h:] * c + x[:, :h] * s], -1)


def norm_rope(y, pos, Hq, H, d, q_gain=None, k_gain=None, eps=1e-6, sections=None, grads=None):
    """y [T, N] -> dict with q, k, v, rstd, or with grads = (dq, dk, dv) dy, dq_gain, dk_gain."""
    y = np.asarray(y, np.float64)
    T = y.shape[0]
    ang = angles(pos, d, sections=sections)
    heads, rstd, dy = [], [], []
    dgain = np.zeros((2, d))
    for h in range(Hq + H):
        x = y[:, h * d:(h + 1) * d]
        gain = (q_gain, k_gain)[h >= Hq]
        gain = np.ones(d) if gain is None else np.asarray(gain, np.float64)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        rstd.append(r[:, 0])
        heads.append(rotate(x * r * gain, ang))
        if grads is not None:
            g = rotate(np.asarray(grads[0][h] if h < Hq else grads[1][h - Hq], np.float64), ang, back=True)
            dgain[int(h >= Hq)] += (g * x * r).sum(0)
            g = g * gain
            dy.append(r * (g - x * r * (g * x * r).mean(-1, keepdims=True)))
    v = y[:, (Hq + H) * d:].reshape(T, H, D_V).transpose(1, 0, 2)
    if grads is None:
        return dict(q=np.stack(heads[:Hq]), k=np.stack(heads[Hq:]), v=v, rstd=np.stack(rstd))
    dv = np.asarray(grads[2], np.float64).transpose(1, 0, 2).reshape(T, H * D_V)
    return dict(dy=np.concatenate(dy + [dv], 1), dq_gain=dgain[0], dk_gain=dgain[1])
