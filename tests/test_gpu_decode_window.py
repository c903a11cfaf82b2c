"""Single-token attention under a window over the paged cache, against the
oracle of the whole attention on the slots that are seen (bounds as in the
tests of the attention without a window)."""

import numpy as np
import pytest
import torch

import synth
from oracle import cache_oracle as co
from test_gpu_cache import DEV, _normal, host, make_cache, qk, same  # noqa: F401

pytestmark = pytest.mark.gpu


def narrowed(c, window, sinks):
    """The cache's dict with only the slots that are seen, in order, and their places."""
    page = c["k"].shape[2]
    keep = [[i for i in range(n) if i >= n - window or i < sinks] for n in c["lengths"]]
    B, most = len(keep), max(1, max(len(x) for x in keep))
    out = {}
    for name in ("k", "v", "k_scale", "v_scale", "weight"):
        x = c[name]
        if x is None:
            out[name] = None
            continue
        y = np.zeros((B,) + (x.shape[1], most) + x.shape[3:], x.dtype)      # one page a sequence
        for b, slots in enumerate(keep):
            for j, i in enumerate(slots):
                y[b, :, j] = x[c["table"][b, i // page], :, i % page]
        out[name] = y
    return dict(out, table=np.arange(B)[:, None], lengths=np.array([len(x) for x in keep])), keep


#  Hq, H, d, page, fp8, lengths, window, sinks
CASES = [
    (2, 2, 96, 64, False, [0, 1, 5, 64, 200], 1, 0),
    (2, 2, 96, 64, False, [0, 1, 5, 64, 200], 16, 0),
    (6, 6, 96, 64, False, [130, 131, 700, 17], 33, 4),
    (6, 6, 96, 32, True, [130, 131, 700, 17], 33, 4),
    (4, 1, 64, 16, False, [300, 20, 0, 47, 48, 49], 40, 9),
    (4, 1, 64, 16, True, [300, 20, 0, 47, 48, 49, 65], 40, 9),
    (6, 1, 128, 128, False, [500, 129], 100, 33),
    (6, 1, 128, 256, True, [500, 129, 600], 100, 33),
    (24, 2, 96, 64, False, [333, 64], 65, 1),
    (24, 2, 96, 64, True, [333, 64], 65, 1),
    (1, 1, 96, 16, False, [5000, 31], 4000, 2),
    (2, 1, 96, 64, True, [3000], 31, 500),
    (2, 2, 64, 64, False, [100, 90], 1000, 5),
    (1, 1, 128, 64, False, [257] * 40, 250, 6),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("Hq,H,d,page,fp8,lens,window,sinks", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{'e4m3' if c[4] else 'bf16'}-w{c[6]}-s{c[7]}" for c in CASES])
def test_window(qk, Hq, H, d, page, fp8, lens, window, sinks, accumulate):   # noqa: F811
    cache, _ = make_cache(qk, lens, H, d, page, fp8, seed=d + window)
    B = len(lens)
    # what is not seen is poison, too
    for b, n in enumerate(lens):
        for i in range(n):
            if i < n - window and i >= sinks:
                p, r = cache.table[b, i // page].item(), i % page
                for t in (cache.k, cache.v):
                    t[p, :, r] = 0x7F if fp8 else float("nan")
                for t in (cache.k_scale, cache.v_scale):
                    if t is not None:
                        t[p, :, r] = float("nan")
    q = _normal((Hq, B, d), 3)
    before = host(cache)
    small, keep = narrowed(before, window, sinks)
    scale = d ** -0.5
    ra, rlse, p, absa, size = co.decode_attention(small, synth.to_numpy_f32(q), scale)
    ws = qk.new_cache_workspace(cache, Hq)
    a, lse = qk.decode_attention(q.to(DEV), cache, accumulate=accumulate, ws=ws, window=window, sinks=sinks)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    a, lse = synth.to_numpy_f32(a).reshape(ra.shape), lse.cpu().numpy()
    delta = (d + 8) * 2.0 ** -23 * size
    bound = 2.0 ** -8 * np.abs(ra) + (2.0 ** -8 + 2 * delta[..., None] + 2.0 ** -20) * absa
    assert (np.abs(a - ra) <= bound).all(), np.abs(a - ra).max()
    none = np.isinf(rlse)
    same(lse[none], rlse[none], "lse of empty sequences")
    assert (np.abs(lse - rlse)[~none] <= (delta + 2.0 ** -20 * (1 + np.abs(rlse)))[~none]).all()
    after = host(cache)
    want, err = before["weight"].astype(np.float64), np.zeros(before["weight"].shape)
    if accumulate:
        G = Hq // H
        for b, slots in enumerate(keep):
            for h in range(H):
                for j, i in enumerate(slots):
                    at = before["table"][b, i // page], h, i % page
                    s = sum(p[b][h * G + g][j] for g in range(G))
                    err[at] = max((2 * delta[b, h * G + g] + 2.0 ** -20) for g in range(G)) * s + 2.0 ** -22 * abs(want[at] + s)
                    want[at] += s
    assert (np.abs(after["weight"] - want) <= err)[~np.isnan(want)].all()
    same(np.isnan(after["weight"]), np.isnan(want), "weights of slots that are not live")
    for name in ("k", "v", "k_scale", "v_scale", "lengths"):
        if before[name] is not None:
            same(after[name], before[name], name)


def test_a_window_of_the_whole_cache_is_no_window(qk):   # noqa: F811
    cache, _ = make_cache(qk, [100, 64, 1], 2, 96, 64, False)
    q = _normal((2, 3, 96), 3).to(DEV)
    a, lse = qk.decode_attention(q, cache)
    b, lsb = qk.decode_attention(q, cache, window=2 ** 40, sinks=2 ** 40)
    assert torch.equal(a, b) and torch.equal(lse, lsb)


def test_captured_window(qk):   # noqa: F811
    cache, _ = make_cache(qk, [700, 64, 0], 2, 96, 64, True)
    q = _normal((2, 3, 96), 3).to(DEV)
    a, lse = qk.decode_attention(q, cache, window=100, sinks=3)
    out, ws = (torch.empty_like(a), torch.empty_like(lse)), qk.new_cache_workspace(cache, 2)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qk.decode_attention(q, cache, window=100, sinks=3, out=out, ws=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out[0]) and torch.equal(lse, out[1])
