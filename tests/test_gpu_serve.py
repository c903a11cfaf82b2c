"""The serving example: projection, append, attention, output projection and
eviction together, the attention checked against float64 over what the
projection has given, step for step."""

import os
import sys

import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
f32 = synth.to_numpy_f32


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_packed_reduced_gb300 import build as b
    b.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import serve_layer
    return serve_layer


def _held(x, fp8):
    """Rows as the cache holds them."""
    if not fp8:
        return f32(x.cpu()).astype(np.float64)
    rows = f32(x.cpu())
    out = np.empty(rows.shape)
    for i in np.ndindex(rows.shape[:-1]):
        codes, s, _ = oracle.quantize(rows[i])
        out[i] = oracle.dequantize(codes, s)
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("budget", [0, 70])
def test_layer_serves(example, fp8, budget):
    D, H, prompts = 768, 6, [33, 0, 60]
    B = len(prompts)
    w = synth.forward_inputs(synth.Shape(sum(prompts), D, H), seed=1, device=DEV)
    Wo = synth.oproj_inputs(1, D, H * 128, device=DEV)["Wo"]
    layer = example.ServingLayer(w["Wq"], w["Wk"], w["Wv"], Wo, H, B, 512, fp8=fp8, budget=budget, recent=16)
    _, k, v = layer.prefill(w["x"], prompts)
    at = np.cumsum([0, *prompts])
    keys, vals = _held(k, fp8), _held(v, fp8)
    seqs = [(keys[:, at[b]:at[b + 1]], vals[:, at[b]:at[b + 1]]) for b in range(B)]
    weights = [np.zeros((H, n)) for n in prompts]
    places = [np.tile(np.arange(n), (H, 1)) for n in prompts]    # tokens (by position) in the slots of every head
    g = torch.Generator().manual_seed(5)
    evicted = 0
    for step in range(150):
        before = layer.held
        x = torch.randn((B, D), generator=g).to(torch.bfloat16).to(DEV)
        _, a, (q, k, v) = layer.step(x)
        if layer.held != before + 1:          # the layer has evicted first
            evicted += 1
            for b in range(B):
                n = places[b].shape[1]
                if n > budget:
                    kept = [oracle.cache_oracle.evict_slots(weights[b][h], places[b][h], budget, 16) for h in range(H)]
                    places[b] = np.stack([places[b][h][kept[h]] for h in range(H)])
                    weights[b] = np.stack([weights[b][h][kept[h]] for h in range(H)])
        kk, vv, qq = _held(k, fp8), _held(v, fp8), f32(q.cpu()).astype(np.float64)
        got = f32(a.cpu()).reshape(B, H, 128)
        have = layer.cache.lengths.tolist()
        for b in range(B):
            seqs[b] = tuple(np.concatenate([s, new[:, b:b + 1]], 1) for s, new in zip(seqs[b], (kk, vv)))
            n = seqs[b][0].shape[1]
            places[b] = np.concatenate([places[b], np.full((H, 1), n - 1)], 1)
            assert have[b] == places[b].shape[1]
            weights[b] = np.concatenate([weights[b], np.zeros((H, 1))], 1)
            for h in range(H):
                ks, vs = seqs[b][0][h][places[b][h]], seqs[b][1][h][places[b][h]]
                s = ks @ qq[h, b] * 96 ** -0.5
                p = np.exp(s - s.max())
                p /= p.sum()
                ref, size = p @ vs, p @ np.abs(vs)
                delta = 104 * 2.0 ** -23 * (np.abs(ks) @ np.abs(qq[h, b])).max() * 96 ** -0.5
                bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * delta + 2.0 ** -20) * size
                assert (np.abs(got[b, h] - ref) <= bound).all(), (step, b, h)
        if budget:   # the weights as the layer has them, so that near-ties of sums cannot part the two
            table, pool = layer.cache.table.cpu().numpy(), layer.cache.weight.cpu().numpy()
            for b in range(B):
                slot = np.arange(have[b])
                now = pool[table[b][slot // 64], :, slot % 64].T
                weights[b] = now
    # 60 + 150 tokens outgrow the 192 slots that the layer has for a budget of 70
    assert evicted == (1 if budget else 0)
    assert example.qk.poll_device_status(layer.ws) == (0, 0)
