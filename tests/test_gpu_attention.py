"""Causal attention over packed sequences on the GPU, through the binding,
against the float64 oracle.

Bounds, fixed by the arithmetic before the first run: the forward's as in the
single-token attention's tests (probabilities rounded to bf16 for the product
with v, 2^-8 relative; scores off by delta = (d + 8) 2^-23 scale sum |q k|):
  |a - ref|   <= 2^-8 |ref| + (2^-8 + 2 delta + 2^-20) sum p |v|
  |lse - ref| <= delta + 2^-20 (1 + |ref|)
the gradients' as written out in oracle.attention_oracle.gradient_bounds."""

import threading

import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import attention_oracle as ao
from helpers import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
f32 = synth.to_numpy_f32


@pytest.fixture(scope="module")
def qk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_packed_reduced_gb300 import build as b
    b.build()
    import fp8_packed_reduced_gb300 as pkg
    pkg.lib()
    return pkg


def _normal(shape, seed, std=1.0):
    return synth._normal(shape, std, seed)


def inputs(Hq, H, T, d, seed=0):
    """q, k with some strong scores; da."""
    q, k, v, da = _normal((Hq, T, d), seed), _normal((H, T, d), seed + 1), _normal((H, T, 128), seed + 2), _normal((T, Hq * 128), seed + 3)
    k[:, ::13] = q[::Hq // H, ::13] * 0.5 + k[:, ::13] * 0.5
    return q, k, v, da


def gpu(*ts):
    return [t.to(DEV).contiguous() for t in ts]


def offsets(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)


def check_forward(a, lse, f, d, name=""):
    delta = (d + 8) * 2.0 ** -23 * f["score"]
    rows = delta.T.repeat(128, -1)
    err = np.abs(f32(a) - f["a"]) - (2.0 ** -8 * np.abs(f["a"]) + (2.0 ** -8 + 2 * rows + 2.0 ** -20) * f["pv"])
    assert err.max() <= 0, f"{name} a: {err.max()} over the bound at {np.unravel_index(err.argmax(), err.shape)}"
    none, got = np.isinf(f["lse"]), lse.cpu().numpy()
    np.testing.assert_array_equal(got[none], f["lse"][none])
    err = np.abs(got[~none] - f["lse"][~none]) - (delta + 2.0 ** -20 * (1 + np.abs(f["lse"])))[~none]
    assert err.size == 0 or err.max() <= 0, f"{name} lse: {err.max()} over the bound"


def check_backward(g, f, b):
    for n in ("dq", "dk", "dv"):
        err = np.abs(f32(g[n]) - f[n]) - b[n]
        assert err.max() <= 0, f"{n}: {err.max()} over the bound at {np.unravel_index(err.argmax(), err.shape)}"
        assert np.isfinite(f32(g[n])).all()


#  Hq, H, d, T, cu, window, sinks
CASES = [
    (1, 1, 96, 1, None, None, 0),
    (2, 1, 64, 2, [0, 1, 2], 1, 0),
    (2, 2, 96, 67, None, None, 0),
    (3, 1, 128, 127, [0, 127], None, 0),
    (2, 2, 96, 128, None, 32, 0),
    (4, 2, 64, 129, [0, 1, 1, 129], None, 0),
    (2, 1, 96, 255, [0, 100, 255], 17, 3),
    (1, 1, 128, 256, None, 128, 4),
    (6, 6, 96, 257, [0, 256, 257], None, 0),
    (2, 2, 64, 300, [3, 150, 150, 297], 64, 1),
    (8, 1, 96, 333, [0, 5, 6, 130, 333], None, 0),
    (2, 1, 128, 385, None, 1, 0),
    (2, 1, 96, 385, None, 1, 4),
    (2, 2, 96, 511, [0, 500], 100, 300),
    (1, 1, 96, 640, None, 129, 130),
    (3, 3, 128, 513, [0, 129, 513], 127, 1),
    (2, 1, 64, 777, [0, 0, 0, 777, 777], 255, 8),
    (2, 1, 96, 900, [0, 260, 900], 300, 257),
    (16, 2, 64, 200, [0, 64, 128, 192], 5000, 0),
    (2, 2, 128, 1100, None, None, 0),
    (1, 1, 64, 1300, None, 640, 16),
]
IDS = ["-".join(str(x) for x in c).replace(" ", "") for c in CASES]


@pytest.mark.parametrize("Hq,H,d,T,cu,window,sinks", CASES, ids=IDS)
def test_forward_and_backward(qk, Hq, H, d, T, cu, window, sinks):
    q, k, v, da = inputs(Hq, H, T, d, seed=T)
    f, b = ao.gradient_bounds(f32(q), f32(k), f32(v), f32(da), cu, window, sinks)
    Q, K, V, DA = gpu(q, k, v, da)
    C = offsets(cu)
    ws = qk.new_attention_workspace(T, Hq)
    a, lse = qk.attention_forward(Q, K, V, C, window, sinks, ws=ws)
    check_forward(a, lse, f, d)
    g = qk.attention_backward(DA, Q, K, V, a, lse, C, window, sinks, ws=ws)
    check_backward(g, f, b)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    # the same on every run, whatever was in the outputs
    a2, l2 = qk.attention_forward(Q, K, V, C, window, sinks, out=(torch.full_like(a, float("nan")), torch.full_like(lse, 3)))
    g2 = qk.attention_backward(DA, Q, K, V, a, lse, C, window, sinks,
                               out={n: torch.full_like(x, float("nan")) for n, x in g.items()})
    assert torch.equal(a, a2) and torch.equal(lse, l2) and all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("B", [50, 700])
def test_many_short_sequences(qk, d, B):
    lens = [(7 * i) % 23 if i % 5 else 0 for i in range(B)]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T = cu[-1] + 9
    q, k, v, da = inputs(2, 1, T, d, seed=B)
    f, b = ao.gradient_bounds(f32(q), f32(k), f32(v), f32(da), cu, 6, 2)
    Q, K, V, DA = gpu(q, k, v, da)
    a, lse = qk.attention_forward(Q, K, V, offsets(cu), 6, 2)
    check_forward(a, lse, f, d)
    check_backward(qk.attention_backward(DA, Q, K, V, a, lse, offsets(cu), 6, 2), f, b)


@pytest.mark.parametrize("d,window,sinks", [(64, None, 0), (96, 100, 3), (128, 33, 260), (96, 1, 0)])
def test_more_tiles_than_multiprocessors(qk, d, window, sinks):
    """Ragged sequences in more tiles than the GPU has multiprocessors, so that
    blocks take several in turn; rows of no sequence before and behind them."""
    lens = [1 + (37 * i) % 413 if i % 7 else 0 for i in range(160)]
    cu = (300 + np.concatenate([[0], np.cumsum(lens)])).tolist()
    T, Hq = cu[-1] + 700, 2
    assert T // 256 * Hq > 190
    q, k, v, da = inputs(Hq, 1, T, d, seed=d)
    f, b = ao.gradient_bounds(f32(q), f32(k), f32(v), f32(da), cu, window, sinks)
    Q, K, V, DA = gpu(q, k, v, da)
    ws = qk.new_attention_workspace(T, Hq)
    a, lse = qk.attention_forward(Q, K, V, offsets(cu), window, sinks, ws=ws)
    check_forward(a, lse, f, d)
    g = qk.attention_backward(DA, Q, K, V, a, lse, offsets(cu), window, sinks, ws=ws)
    check_backward(g, f, b)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    for _ in range(3):   # the same on every run, and the workspace is left as it has to be
        a2, l2 = qk.attention_forward(Q, K, V, offsets(cu), window, sinks, ws=ws)
        g2 = qk.attention_backward(DA, Q, K, V, a, lse, offsets(cu), window, sinks, ws=ws)
        assert torch.equal(a, a2) and torch.equal(lse, l2) and all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("scale", [1e-6, 0.02, 3.0])
def test_scales(qk, scale):
    """Flat, ordinary and very peaked probabilities."""
    q, k, v, da = inputs(2, 1, 200, 96, seed=4)
    f, b = ao.gradient_bounds(f32(q), f32(k), f32(v), f32(da), [0, 180], 70, 2, scale)
    Q, K, V, DA = gpu(q, k, v, da)
    a, lse = qk.attention_forward(Q, K, V, offsets([0, 180]), 70, 2, scale)
    check_forward(a, lse, f, 96)
    check_backward(qk.attention_backward(DA, Q, K, V, a, lse, offsets([0, 180]), 70, 2, scale), f, b)


def test_scores_that_grow_and_fall(qk):
    """Along the keys: every running maximum is replaced, and the first holds."""
    T, d = 700, 96
    for sign in (1, -1):
        q, k, v, _ = inputs(1, 1, T, d, seed=9)
        q[0] = 1.0
        k[0] = (k[0].float() * 0.1 + sign * torch.linspace(-4, 4, T)[:, None]).to(torch.bfloat16)
        f = ao.attention(f32(q), f32(k), f32(v))
        check_forward(*qk.attention_forward(*gpu(q, k, v)), f, d, str(sign))


def test_exact_zeros(qk):
    """Tokens that see only themselves: a = v, and nothing reaches q and k."""
    for T, cu, window in ((300, None, 1), (64, list(range(65)), None)):
        q, k, v, da = gpu(*inputs(2, 1, T, 96, seed=1))
        a, lse = qk.attention_forward(q, k, v, offsets(cu), window)
        assert torch.equal(a.view(T, 2, 128), v[0][:, None].expand(T, 2, 128))
        g = qk.attention_backward(da, q, k, v, a, lse, offsets(cu), window)
        assert not g["dq"].any() and not g["dk"].any()


BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("bad", BAD, ids=str)
@pytest.mark.parametrize("which", ["q", "k", "v", "da", "all"])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_what_is_not_seen_has_no_part(qk, bad, which, d):
    """Bad values in one token (and in the rows of no sequence) reach the tokens
    that see it, or that it sees, and no others."""
    Hq, H, T, cu, window, sinks = 2, 1, 420, [0, 130, 400], 50, 2
    at = (131, 250)      # a sink of the second sequence; a token that leaves the window
    q, k, v, da = inputs(Hq, H, T, d, seed=6)
    f, b = ao.gradient_bounds(f32(q), f32(k), f32(v), f32(da), cu, window, sinks)
    hit = {n: np.zeros(T, bool) for n in ("a", "dq", "dkv")}
    seen = np.zeros((T, T), bool)
    for s, e in ao.spans(cu, T):
        seen[s:e, s:e] = ao.seen(e - s, window, sinks)
    for t in at[1:] if which in ("k", "v") else at:
        for n, x in (("q", q), ("k", k), ("v", v)):
            if which in (n, "all"):
                x[0, t] = bad
        if which in ("da", "all"):
            da[t] = bad
    for n, x in (("q", q), ("k", k), ("v", v)):
        x[:, 400:] = bad
    da[400:] = bad
    touched = at[1:] if which in ("k", "v") else at
    for t in touched:
        rows = seen[:, t] if which in ("k", "v", "all") else np.eye(T, dtype=bool)[t]
        if which != "da":
            hit["a"] |= rows
        hit["dq"] |= rows
        hit["dkv"] |= seen[rows].any(0)
    Q, K, V, DA = gpu(q, k, v, da)
    a, lse = qk.attention_forward(Q, K, V, offsets(cu), window, sinks)
    ok = ~hit["a"]
    delta = (d + 8) * 2.0 ** -23 * f["score"].T.repeat(128, -1)
    err = np.abs(f32(a) - f["a"]) - (2.0 ** -8 * np.abs(f["a"]) + (2.0 ** -8 + 2 * delta + 2.0 ** -20) * f["pv"])
    assert (err[ok] <= 0).all()
    assert (f32(a)[400:] == 0).all() and (lse[:, 400:] == -float("inf")).all()
    g = qk.attention_backward(DA, Q, K, V, a, lse, offsets(cu), window, sinks)
    for n, rows in (("dq", ~hit["dq"]), ("dk", ~hit["dkv"]), ("dv", ~hit["dkv"])):
        assert (np.abs(f32(g[n]) - f[n])[:, rows] <= b[n][:, rows]).all(), n
        assert not g[n][:, 400:].any(), n
    if which == "v" and bad != bad:
        t = at[1]
        assert np.isnan(f32(a)[t:t + window]).all() and np.isnan(f32(g["dq"])[:, t + 1:t + window]).all()


def test_bad_offsets_are_recorded(qk):
    q, k, v, da = gpu(*inputs(2, 1, 300, 96, seed=2))
    ws = qk.new_attention_workspace(300, 2)
    for cu, kid in (([0, 400], 18), ([-5, 300], 18), ([0, 200, 100, 300], 18)):
        a, lse = qk.attention_forward(q, k, v, offsets(cu), ws=ws)
        assert qk.poll_device_status(ws)[0] == qk.ERR_DEVICE_INPUT
        qk.attention_backward(da, q, k, v, a, lse, offsets(cu), ws=ws)
        assert qk.poll_device_status(ws)[0] == qk.ERR_DEVICE_INPUT
        if cu != [0, 200, 100, 300]:      # the nearer end
            f = ao.attention(f32(q.cpu()), f32(k.cpu()), f32(v.cpu()), cu)
            check_forward(a, lse, f, 96)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    qk.attention_forward(q, k, v, offsets([0, 400]))
    assert qk.poll_cache_status()[0] == qk.ERR_DEVICE_INPUT


def test_no_tokens(qk):
    q, k, v = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((2, 0, 96), (1, 0, 96), (1, 0, 128)))
    a, lse = qk.attention_forward(q, k, v)
    assert a.shape == (0, 256) and lse.shape == (2, 0)
    g = qk.attention_backward(a, q, k, v, a, lse, offsets([0, 0]))
    assert g["dq"].shape == (2, 0, 96)
    q, k, v, da = gpu(*inputs(2, 1, 70, 96))
    a, lse = qk.attention_forward(q, k, v, offsets([0, 0, 0]))
    assert not a.any() and (lse == -float("inf")).all()
    g = qk.attention_backward(da, q, k, v, a, lse, offsets([0, 0, 0]))
    assert not any(x.any() for x in g.values())


def test_captured_calls_and_side_streams(qk):
    Hq, H, T, d, cu = 4, 2, 500, 96, [0, 200, 500]
    q, k, v, da = gpu(*inputs(Hq, H, T, d, seed=3))
    C = offsets(cu)
    a, lse = qk.attention_forward(q, k, v, C, 64, 2)
    g = qk.attention_backward(da, q, k, v, a, lse, C, 64, 2)
    ws = qk.new_attention_workspace(T, Hq)
    oa, ol, og = torch.empty_like(a), torch.empty_like(lse), {n: torch.empty_like(x) for n, x in g.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qk.attention_forward(q, k, v, C, 64, 2, ws=ws, out=(oa, ol))
        qk.attention_backward(da, q, k, v, oa, ol, C, 64, 2, ws=ws, out=og)
    with pytest.raises(ValueError, match="captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            qk.attention_forward(q, k, v, C, 64, 2, out=(oa, ol))
    for seed in (3, 8):
        new = gpu(*inputs(Hq, H, T, d, seed=seed))
        for old, x in zip((q, k, v, da), new):
            old.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        a, lse = qk.attention_forward(q, k, v, C, 64, 2)
        g = qk.attention_backward(da, q, k, v, a, lse, C, 64, 2)
        assert torch.equal(a, oa) and torch.equal(lse, ol) and all(torch.equal(g[n], og[n]) for n in g)
    side, got = [torch.cuda.Stream() for _ in range(3)], [None] * 3
    torch.cuda.synchronize()

    def go(i):
        with torch.cuda.stream(side[i]):
            for _ in range(4):
                x = qk.attention_forward(q, k, v, C, 64, 2)
                got[i] = qk.attention_backward(da, q, k, v, *x, C, 64, 2)
    threads = [threading.Thread(target=go, args=(i,)) for i in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert all(torch.equal(g[n], x[n]) for x in got for n in g)


def test_between_the_projections(qk):
    """As they are used: packed projection, attention, output projection and
    back, and the same prompts' last tokens through the cache."""
    T, D, H, d, cu, window, sinks = 640, 768, 6, 96, [0, 400, 640], 200, 4
    s = synth.Shape(T=T, D=D, H=H, d_qk=d, d_v=128, seq_len=T)
    inp = synth.forward_inputs(s, seed=1)
    pos = torch.cat([torch.arange(400), torch.arange(240)]).to(torch.int32).to(DEV)
    W8, W8T, sw = qk.quantize_bank([tuple(inp[n].to(DEV) for n in ("Wq", "Wk", "Wv"))], H, d)
    table = qk.build_rope_table(T, d)
    op = synth.oproj_inputs(T, D, H * 128, seed=2)
    Wo8, Wo8T, so = qk.quantize_weight([op["Wo"].to(DEV)])
    C = offsets(cu)
    q, k, v, saved = qk.forward(inp["x"].to(DEV), pos, W8[0], sw[0:1], H, table, d)
    a, lse = qk.attention_forward(q, k, v, C, window, sinks)
    out, a8, sa = qk.oproj_forward(a, Wo8[0], so[0:1])
    og = qk.oproj_backward(op["dout"].to(DEV), Wo8T[0], so[0:1], a8, sa)
    g = qk.attention_backward(og["da"], q, k, v, a, lse, C, window, sinks)
    grads = qk.backward(g["dq"], g["dk"], g["dv"], saved, W8T[0], sw[0:1], table)
    f, b = ao.gradient_bounds(f32(q), f32(k), f32(v), f32(og["da"]), cu, window, sinks)
    check_forward(a, lse, f, d)
    check_backward(g, f, b)
    # the whole way from the attention's gradients as they are
    bw = oracle.backward(f32(g["dq"]), f32(g["dk"]), f32(g["dv"]), f32(saved.q), f32(saved.k), saved.rstd.cpu().numpy(),
                         pos.cpu().numpy(), W8[0].cpu().numpy(), sw[0].item(), saved.x8.cpu().numpy(),
                         saved.x_scale.item(), H, d, 128)
    # (a sequence's first tokens have few others to share da with: dx is as heavy-tailed
    # as its largest value 4 beside an rms of 0.3, and rounding that to bf16 alone is off
    # by up to 4 * 2^-8 = 0.016 > 2e-2 * 0.3)
    assert np.abs(bw["dX"]).max() * 2.0 ** -8 > 2e-2 * np.sqrt((bw["dX"] ** 2).mean())
    assert_close(f32(grads["dx"]), bw["dX"], "dx", bf16_rounding=True)
    assert_close(f32(grads["dW"]), bw["dW"], "dW", bf16_rounding=True)
    # serving: the window of the cache's last token is that of the prompt's
    cache = qk.new_cache(2, 400, H, d)
    qk.cache_append(cache, k, v, pos, cu=C)
    last = [399, 639]
    a1, lse1 = qk.decode_attention(q[:, last].contiguous(), cache, window=window, sinks=sinks)
    part = {n: x for n, x in f.items()}
    part.update(a=f["a"][last], pv=f["pv"][last], lse=f["lse"][:, last], score=f["score"][:, last])
    check_forward(a1, lse1.t(), part, d, "cache")
