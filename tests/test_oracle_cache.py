"""Pins of the cache oracle, against something other than itself (CPU)."""

import numpy as np
import torch

from oracle import cache_oracle as co


def _cache(rng, lens, H=2, d=64, page=16, cap=80):
    B, pages = len(lens), cap // page
    P = B * pages + 2
    return dict(k=rng.standard_normal((P, H, page, d)), v=rng.standard_normal((P, H, page, 128)),
                pos=rng.integers(0, 1000, (P, H, page)), weight=rng.random((P, H, page)),
                table=rng.permutation(P)[:B * pages].reshape(B, pages), lengths=np.array(lens))


def test_decode_is_dense_attention():
    rng = np.random.default_rng(0)
    c = _cache(rng, [37, 0, 1])
    q = rng.standard_normal((4, 3, 64))
    a, lse, p, _, _ = co.decode_attention(c, q, 0.125)
    for b, n in enumerate(c["lengths"]):
        for hq in range(4):
            if n == 0:
                assert (a[b, hq] == 0).all() and lse[b, hq] == -np.inf
                continue
            k = c["k"][c["table"][b]].transpose(1, 0, 2, 3).reshape(2, -1, 64)[hq // 2, :n]
            v = c["v"][c["table"][b]].transpose(1, 0, 2, 3).reshape(2, -1, 128)[hq // 2, :n]
            ref = torch.nn.functional.scaled_dot_product_attention(
                *(torch.from_numpy(x)[None] for x in (q[hq, b:b + 1], k, v)), scale=0.125)[0, 0].numpy()
            np.testing.assert_allclose(a[b, hq], ref, rtol=1e-12, atol=1e-13)
            np.testing.assert_allclose(p[b][hq].sum(), 1, rtol=1e-12)


def test_append_then_read_back():
    rng = np.random.default_rng(1)
    c = _cache(rng, [3, 0, 40])
    cu = np.array([0, 14, 14, 20])
    k, v = rng.standard_normal((2, 20, 64)), rng.standard_normal((2, 20, 128))
    old = co.live_rows(c, 0, 1)[0]
    c["lengths"] = co.cache_append(c, k, v, np.arange(20), cu)
    assert list(c["lengths"]) == [17, 0, 46]
    got = co.live_rows(c, 0, 1)[0]
    np.testing.assert_array_equal(got[:3], old)
    np.testing.assert_array_equal(got[3:], k[1, :14])
    np.testing.assert_array_equal(co.live_rows(c, 2, 0)[1][40:], v[0, 14:20])


def test_evict_keeps_the_best_and_moves_little():
    rng = np.random.default_rng(2)
    for _ in range(200):
        n = int(rng.integers(2, 60))
        budget = int(rng.integers(1, n))
        recent = int(rng.integers(0, budget + 1))
        w = rng.integers(0, 6, n) / 2.0           # many ties
        pos = rng.permutation(n) + 5
        got = co.evict_slots(w, pos, budget, recent)
        assert len(set(got)) == budget
        # the set: newest `recent` positions, then stable order of falling weight
        newest = set(np.argsort(-pos)[:recent].tolist())
        rest = [i for i in np.argsort(-w, kind="stable").tolist() if i not in newest]
        assert set(got) == newest | set(rest[:budget - recent])
        # kept slots below the budget stay, the others fill the holes in order
        assert all(g == j or g >= budget for j, g in enumerate(got))
        moved = [g for j, g in enumerate(got) if g != j]
        assert moved == sorted(moved)
