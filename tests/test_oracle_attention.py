"""The float64 oracle of the attention and of the split, norm and rotation:
against differences, and against the other oracles where they meet."""

import numpy as np
import pytest

import oracle
from oracle import attention_oracle as ao


def _inputs(Hq, H, T, d, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((Hq, T, d)), r.standard_normal((H, T, d)), r.standard_normal((H, T, 128)), r.standard_normal((T, Hq * 128))


def test_what_a_token_sees():
    s = ao.seen(6, 2, 1)
    assert [np.flatnonzero(r).tolist() for r in s] == [[0], [0, 1], [0, 1, 2], [0, 2, 3], [0, 3, 4], [0, 4, 5]]
    assert ao.seen(5, None, 3).tolist() == np.tril(np.ones((5, 5), bool)).tolist()
    assert ao.seen(4, 1, 0).tolist() == np.eye(4, dtype=bool).tolist()


@pytest.mark.parametrize("window,sinks", [(None, 0), (3, 0), (2, 2), (1, 0)])
def test_gradients_against_differences(window, sinks):
    q, k, v, da = _inputs(4, 2, 9, 64)
    cu = [0, 4, 4, 8]
    f = ao.attention(q, k, v, cu, window, sinks, da=da)
    r = np.random.default_rng(5)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        step = r.standard_normal(x.shape)
        at = dict(q=q, k=k, v=v)
        ends = []
        for h in (1e-5, -1e-5):
            at[name[1]] = x + h * step
            ends.append((ao.attention(at["q"], at["k"], at["v"], cu, window, sinks)["a"] * da).sum())
        slope = (ends[0] - ends[1]) / 2e-5
        np.testing.assert_allclose((f[name] * step).sum(), slope, rtol=1e-6, atol=1e-7)


def test_rows_of_no_sequence():
    q, k, v, da = _inputs(2, 1, 7, 64)
    f = ao.attention(q, k, v, [1, 3, 5], da=da)
    for t in (0, 5, 6):
        assert (f["a"][t] == 0).all() and (f["lse"][:, t] == -np.inf).all()
        assert (f["dq"][:, t] == 0).all() and (f["dk"][:, t] == 0).all() and (f["dv"][:, t] == 0).all()


def test_gradient_bounds_hold_for_rounded_operands():
    """The bounds cover what they are for: probabilities, ds and results rounded to bf16."""
    def bf16(x):
        return oracle.to_bf16(np.float32(x)).astype(np.float64)
    q, k, v, da = (bf16(x) for x in _inputs(2, 1, 40, 96, 3))
    f, b = ao.gradient_bounds(q, k, v, da, None, 16, 2)
    ok, scale = ao.seen(40, 16, 2), 96 ** -0.5
    dk, dv = np.zeros((40, 96)), np.zeros((40, 128))
    for h in range(2):
        x = np.where(ok, scale * q[h] @ k[0].T, -np.inf)
        p = np.exp(x - f["lse"][h][:, None])
        g = da[:, h * 128:(h + 1) * 128]
        ds = bf16(p * (g @ v[0].T - (g * bf16(f["a"][:, h * 128:(h + 1) * 128])).sum(-1, keepdims=True)))
        dk += scale * ds.T @ q[h]
        dv += bf16(p).T @ g
        assert (np.abs(bf16(scale * ds @ k[0]) - f["dq"][h]) <= b["dq"][h]).all()
    assert (np.abs(bf16(dk) - f["dk"][0]) <= b["dk"][0]).all()
    assert (np.abs(bf16(dv) - f["dv"][0]) <= b["dv"][0]).all()


@pytest.mark.parametrize("d", [64, 96, 128])
def test_norm_rope_is_the_projections_epilogue(d):
    r = np.random.default_rng(1)
    y, pos = r.standard_normal((5, 2 * 2 * d + 2 * 128)), np.array([0, 3, 8, 1, 100])
    f = ao.norm_rope(y, pos, 2, 2, d)
    for h in range(2):
        for name, col in (("q", h * d), ("k", (2 + h) * d)):
            n, _ = oracle.rms_norm(y[:, col:col + d], 1e-6)
            ang = oracle.rope_angles(pos, d)
            np.testing.assert_allclose(f[name][h], oracle.rope(n, ang), rtol=2e-6, atol=2e-6)


@pytest.mark.parametrize("sections", [None, (8, 24), (4, 14, 14)])
def test_norm_rope_gradients_against_differences(sections):
    r = np.random.default_rng(2)
    Hq, H, d, T = 4, 2, 64, 5
    y = r.standard_normal((T, 6 * d + H * 128))
    pos = r.integers(0, 50, (T,) if sections is None else (len(sections), T))
    qg, kg = r.standard_normal(d), r.standard_normal(d)
    g = r.standard_normal((Hq, T, d)), r.standard_normal((H, T, d)), r.standard_normal((H, T, 128))
    b = ao.norm_rope(y, pos, Hq, H, d, qg, kg, 1e-6, sections, g)

    def loss(y, qg, kg):
        f = ao.norm_rope(y, pos, Hq, H, d, qg, kg, 1e-6, sections)
        return sum((f[n] * x).sum() for n, x in zip("qkv", g))
    for name, i in (("dy", 0), ("dq_gain", 1), ("dk_gain", 2)):
        args = [y, qg, kg]
        step = r.standard_normal(args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * step, args[i] - 1e-5 * step
        np.testing.assert_allclose((b[name] * step).sum(), (loss(*up) - loss(*down)) / 2e-5, rtol=1e-6, atol=1e-6)
