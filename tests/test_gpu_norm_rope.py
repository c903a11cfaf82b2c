"""Split, norm and rotation of a packed projection's rows on the GPU, through the
binding, against the float64 oracle.

Bounds, fixed by the arithmetic (u = 2^-24, half a float32 step): a sum of d
squares and the root leave r off by (d / 2 + 4) u relative, products and the
table's entries (each off by u) 8 u of |x| r |gain| more, and the result is
rounded to bf16, 2^-8 relative:
  |out - ref| <= 2^-8 |ref| + (d / 2 + 12) u (|R| |x r gain|)
The gradient's dot over d columns is off by (d + 8) u of its absolute sum:
  |dx - ref| <= 2^-8 |ref| + r ((d / 2 + 16) u |g gain| + |x r| (2 d + 24) u mean |g gain x r|)
A gain's sum over n = tokens x heads by (n + d + 16) u of the sum of |g x r|."""

import numpy as np
import pytest
import torch

import synth
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
f32 = synth.to_numpy_f32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def qk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_packed_reduced_gb300 import build as b
    b.build()
    import fp8_packed_reduced_gb300 as pkg
    pkg.lib()
    return pkg


def spread(x, ang):
    """|R| |x|: what a rotation of x can reach."""
    x, h = np.abs(x), x.shape[-1] // 2
    c, s = np.abs(np.cos(ang)), np.abs(np.sin(ang))
    return np.concatenate([x[:, :h] * c + x[:, h:] * s, x[:, h:] * c + x[:, :h] * s], -1)


#  Hq, H, d, T, gain, sections, extra columns, positions below
CASES = [
    (1, 1, 64, 1, False, None, 0, 1),
    (6, 6, 96, 1, True, None, 0, 64),
    (6, 6, 96, 333, True, None, 0, 8192),
    (4, 2, 64, 65, True, (8, 24), 8, 100),
    (8, 1, 128, 77, False, (12, 26, 26), 136, 50),
    (3, 3, 96, 40, True, (8, 20, 20), 0, 131072),
    (2, 1, 96, 31, True, (0, 48), 64, 30),
    (2, 1, 128, 1000, True, (64, 0, 0), 0, 1000),
    (16, 8, 64, 5000, True, None, 0, 5000),
    (1, 1, 128, 20000, False, None, 0, 300),
]


@pytest.mark.parametrize("Hq,H,d,T,gain,sections,extra,far", CASES, ids=["-".join(str(x) for x in c[:4]) for c in CASES])
def test_forward_and_backward(qk, Hq, H, d, T, gain, sections, extra, far):
    N, r = (Hq + H) * d + H * 128, np.random.default_rng(T)
    y = synth._normal((T, N + extra), 1.0, T)
    y[T // 2] *= 30
    pos = r.integers(0, far, (T,) if sections is None else (len(sections), T)).astype(np.int32)
    qg, kg = (r.uniform(-2, 2, d).astype(np.float32) for _ in range(2)) if gain else (None, None)
    grads = [synth._normal(s, 0.1, T + i) for i, s in enumerate(((Hq, T, d), (H, T, d), (H, T, 128)))]
    yn = f32(y)[:, :N]
    f = ao.norm_rope(yn, pos, Hq, H, d, qg, kg, 1e-6, sections)
    b = ao.norm_rope(yn, pos, Hq, H, d, qg, kg, 1e-6, sections, [f32(g) for g in grads])
    to = lambda x: None if x is None else torch.from_numpy(x).to(DEV)   # noqa: E731
    Y = y.to(DEV)[:, :N]
    table, P, QG, KG = qk.build_rope_table(far, d), to(pos), to(qg), to(kg)
    ws = qk.new_norm_rope_workspace()
    q, k, v, rstd = qk.norm_rope_forward(Y, P, table, Hq, H, d, QG, KG, sections=sections, ws=ws)
    g = qk.norm_rope_backward(*(x.to(DEV) for x in grads), Y, rstd, P, table, QG, KG, sections, ws=ws)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    ang = ao.angles(pos, d, sections=sections)
    np.testing.assert_allclose(rstd.cpu().numpy(), f["rstd"], rtol=(d / 2 + 4) * U, atol=0)
    assert np.array_equal(f32(v), f["v"].astype(np.float32))
    assert np.array_equal(f32(g["dy"])[:, (Hq + H) * d:], f32(grads[2]).transpose(1, 0, 2).reshape(T, -1))
    sums = np.zeros((2, d))
    for h in range(Hq + H):
        name, i, gn = ("q", h, qg) if h < Hq else ("k", h - Hq, kg)
        gn = np.ones(d) if gn is None else gn.astype(np.float64)
        x, ref = yn[:, h * d:(h + 1) * d].astype(np.float64), f[name][i]
        rs = f["rstd"][h][:, None]
        got = f32((q, k)[h >= Hq][i])
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (d / 2 + 12) * U * spread(x * rs * gn, ang)).all(), (name, i)
        gr = f32(grads[int(h >= Hq)][i]).astype(np.float64)
        gg, xr = spread(gr, ang), np.abs(x * rs)
        sums[int(h >= Hq)] += (gg * xr).sum(0)
        ref, got = b["dy"][:, h * d:(h + 1) * d], f32(g["dy"])[:, h * d:(h + 1) * d]
        err = rs * ((d / 2 + 16) * U * gg * np.abs(gn) + xr * (2 * d + 24) * U * (gg * np.abs(gn) * xr).mean(-1, keepdims=True))
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + err).all(), ("d" + name, i)
    if gain:
        for w, (n, heads) in enumerate((("dq_gain", Hq), ("dk_gain", H))):
            assert (np.abs(g[n].cpu().numpy() - b[n]) <= (T * heads + d + 16) * U * sums[w]).all(), n
    else:
        assert g["dq_gain"] is None and g["dk_gain"] is None
    again = qk.norm_rope_backward(*(x.to(DEV) for x in grads), Y, rstd, P, table, QG, KG, sections)
    assert all(x is None or torch.equal(x, again[n]) for n, x in g.items())


def test_positions_outside_the_table(qk):
    y = synth._normal((4, 2 * 96 + 128), 1.0, 0).to(DEV)
    table, ws = qk.build_rope_table(10, 96), qk.new_norm_rope_workspace()
    pos = torch.tensor([-1, 3, 10, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    q, *_ = qk.norm_rope_forward(y, pos, table, 1, 1, ws=ws)
    assert qk.poll_device_status(ws) == (qk.ERR_DEVICE_INPUT, 22)
    want, *_, rstd = qk.norm_rope_forward(y, pos.clamp(0, 9), table, 1, 1, ws=ws)
    assert torch.equal(q, want) and qk.poll_device_status(ws) == (qk.OK, 0)
    qk.norm_rope_backward(want, want, torch.zeros((1, 4, 128), dtype=torch.bfloat16, device=DEV), y, rstd, pos, table, ws=ws)
    assert qk.poll_device_status(ws) == (qk.ERR_DEVICE_INPUT, 23)


def test_zero_nan_and_infinite_rows_stay_where_they_are(qk):
    Hq, H, d, T = 2, 1, 96, 6
    y = synth._normal((T, 3 * d + 128), 1.0, 0)
    clean, *_ = qk.norm_rope_forward(y.to(DEV), torch.arange(T, dtype=torch.int32, device=DEV), qk.build_rope_table(T, d), Hq, H, d)
    y[1, :d] = 0
    y[2, 5], y[3, 6] = float("nan"), float("inf")
    q, k, v, rstd = qk.norm_rope_forward(y.to(DEV), torch.arange(T, dtype=torch.int32, device=DEV), qk.build_rope_table(T, d), Hq, H, d)
    assert not q[0, 1].any() and abs(rstd[0, 1].item() - 1000) < 1e-3
    assert q[0, 2].isnan().all() and rstd[0, 3] == 0
    assert torch.equal(q[1], clean[1]) and torch.equal(q[0, 4:], clean[0, 4:]) and k.isfinite().all()


def test_no_tokens(qk):
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)   # noqa: E731
    table, pos, gain = qk.build_rope_table(4, 96), torch.empty(0, dtype=torch.int32, device=DEV), torch.ones(96, device=DEV)
    q, k, v, rstd = qk.norm_rope_forward(e(0, 320), pos, table, 1, 1, 96, gain, gain)
    assert q.shape == (1, 0, 96) and rstd.shape == (2, 0)
    g = qk.norm_rope_backward(q, k, v, e(0, 320), rstd, pos, table, gain, gain)
    assert g["dy"].shape == (0, 320) and not g["dq_gain"].any() and not g["dk_gain"].any()


def test_captured(qk):
    Hq, H, d, T = 4, 2, 64, 700
    y = synth._normal((T, 6 * d + H * 128), 1.0, 0).to(DEV)
    pos, table = torch.arange(T, dtype=torch.int32, device=DEV), qk.build_rope_table(T, d)
    gain = torch.rand(d, device=DEV) + 0.5
    f = qk.norm_rope_forward(y, pos, table, Hq, H, d, gain, gain)
    g = qk.norm_rope_backward(*f[:3], y, f[3], pos, table, gain, gain)
    ws = qk.new_norm_rope_workspace()
    of, og = tuple(torch.empty_like(x) for x in f), {n: torch.empty_like(x) for n, x in g.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qk.norm_rope_forward(y, pos, table, Hq, H, d, gain, gain, ws=ws, out=of)
        qk.norm_rope_backward(*of[:3], y, of[3], pos, table, gain, gain, ws=ws, out=og)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(f, of)) and all(torch.equal(g[n], og[n]) for n in g)


def test_a_training_chain(qk):
    """Split, attention, and both gradients back to the packed rows, against
    differences of the whole chain's 64-bit form."""
    Hq, H, d, T, cu, window, sinks = 2, 1, 96, 60, [0, 25, 60], 20, 2
    N = 3 * d + 128
    y, pos = synth._normal((T, N), 1.0, 5), np.concatenate([np.arange(25), np.arange(35)]).astype(np.int32)
    gain = (np.linspace(0.5, 1.5, d).astype(np.float32), np.linspace(1.5, 0.5, d).astype(np.float32))
    da = synth._normal((T, Hq * 128), 1.0, 6)
    Y, P, C = y.to(DEV), torch.from_numpy(pos).to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV)
    G = [torch.from_numpy(x).to(DEV) for x in gain]
    table = qk.build_rope_table(64, d)
    q, k, v, rstd = qk.norm_rope_forward(Y, P, table, Hq, H, d, *G)
    a, lse = qk.attention_forward(q, k, v, C, window, sinks)
    ag = qk.attention_backward(da.to(DEV), q, k, v, a, lse, C, window, sinks)
    g = qk.norm_rope_backward(ag["dq"], ag["dk"], ag["dv"], Y, rstd, P, table, *G)

    def loss(y, qg, kg):
        f = ao.norm_rope(y, pos, Hq, H, d, qg, kg)
        return (ao.attention(f["q"], f["k"], f["v"], cu, window, sinks)["a"] * f32(da)).sum()
    args = [f32(y).astype(np.float64), gain[0].astype(np.float64), gain[1].astype(np.float64)]
    r = np.random.default_rng(0)
    for i, n in enumerate(("dy", "dq_gain", "dk_gain")):
        got = f32(g[n]) if n == "dy" else g[n].cpu().numpy()
        for _ in range(3):
            # along the gradient and across it: what rounds to bf16 is off by 2^-8 of each term
            step = np.sign(got) + r.standard_normal(got.shape)
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + 1e-5 * step, args[i] - 1e-5 * step
            slope = (loss(*up) - loss(*down)) / 2e-5
            # q, k, v, a, p, ds, their gradients and dy: eight roundings of 2^-8
            assert abs((got * step).sum() - slope) <= 8 * 2.0 ** -8 * np.abs(got * step).sum(), n
