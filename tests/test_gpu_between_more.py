"""Norm and rotation where blocks take many chunks of rows, the attention's plan
in replayed graphs, and the calls between the projections mixed with the cache's
on one stream's kept workspace."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def qk():
    from fp8_packed_reduced_gb300 import build as b
    b.build()
    import fp8_packed_reduced_gb300 as pkg
    return pkg


def normal(shape, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def turn(x, cos, sin):
    u, w = x.chunk(2, -1)
    return torch.cat([u * cos - w * sin, w * cos + u * sin], -1)


def size_of_turn(x, cos, sin):
    """The same with every term's size: what float32 may be off by is relative to it."""
    u, w = x.abs().chunk(2, -1)
    return torch.cat([u * cos.abs() + w * sin.abs(), w * cos.abs() + u * sin.abs()], -1)


# tokens that are no multiple of a tile, and more (tile, rows) chunks than blocks on
# the GPU; heads that make chunks of one, of unequal and of whole numbers of rows
@pytest.mark.parametrize("Hq,H,d,T,gain", [(14, 2, 96, 9001, True), (7, 7, 128, 13003, True), (4, 1, 64, 30011, True),
                                           (13, 1, 96, 9001, False)])
def test_norm_rope_with_more_chunks_than_blocks(qk, Hq, H, d, T, gain):
    N = (Hq + H) * d + H * 128
    y = normal((T, N + 24), 1)[:, :N]
    pos = torch.arange(T, dtype=torch.int32, device=DEV) % 1000
    table = qk.build_rope_table(1000, d).to(DEV)
    gains = [torch.linspace(0.5, 1.5, d, device=DEV), torch.linspace(1.5, 0.5, d, device=DEV)] if gain else [None, None]
    q, k, v, rstd = qk.norm_rope_forward(y, pos, table, Hq, H, d, *gains)
    dq, dk, dv = normal((Hq, T, d), 2), normal((H, T, d), 3), normal((H, T, 128), 4)
    g = qk.norm_rope_backward(dq, dk, dv, y, rstd, pos, table, *gains)
    again = qk.norm_rope_backward(dq, dk, dv, y, rstd, pos, table, *gains)
    assert all(torch.equal(g[n], again[n]) for n in g if g[n] is not None)

    entry = table.double()[:, pos.long()]                       # [d / 4, T, 4]: two cosines, two sines
    cos, sin = (entry[..., i:i + 2].permute(1, 0, 2).reshape(T, d // 2) for i in (0, 2))
    rows = y.double()[:, :(Hq + H) * d].reshape(T, Hq + H, d).transpose(0, 1)
    assert torch.equal(v, y[:, (Hq + H) * d:].reshape(T, H, 128).transpose(0, 1))
    dy = g["dy"][:, :(Hq + H) * d].reshape(T, Hq + H, d).transpose(0, 1)
    assert torch.equal(g["dy"][:, (Hq + H) * d:], dv.transpose(0, 1).reshape(T, H * 128))
    for name, part, got, grad, gn, r32 in (("q", slice(0, Hq), q, dq, gains[0], rstd[:Hq]),
                                           ("k", slice(Hq, Hq + H), k, dk, gains[1], rstd[Hq:])):
        x = rows[part]
        w = torch.ones(d, dtype=torch.float64, device=DEV) if gn is None else gn.double()
        r = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        # a sum of d squares, a quotient and a root: within (d / 8 + 8) 2^-24 < 2^-19
        assert ((r32.double()[..., None] - r).abs() <= 2.0 ** -19 * r).all(), name
        n = x * r
        ref = turn(n * w, cos, sin)
        # the result's rounding, and r's and five operations' in float32
        assert ((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -18 * size_of_turn(n * w, cos, sin)).all(), name
        t = turn(grad.double(), cos, -sin)
        ts = size_of_turn(grad.double(), cos, sin)
        dot = (t * w * n).mean(-1, keepdim=True)
        ref = r * (t * w - n * dot)
        size = r * (ts * w + n.abs() * (ts * w * n.abs()).mean(-1, keepdim=True))
        assert ((dy[part].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -17 * size).all(), name
        if gn is not None:
            # A lane adds up no more than three chunks of six rows (18), then lanes (3), warps
            # (4), partials (6 + 2 + 32): fewer than 96 roundings, and 2^-18 of r and the terms'.
            ref, size = (t * n).sum((0, 1)), (ts * n.abs()).sum((0, 1))
            assert ((g["d" + name + "_gain"].double() - ref).abs() <= 2.0 ** -16 * size).all(), name


def test_a_replayed_plan(qk):
    """More tiles than multiprocessors: jobs and counters are made anew by every replay."""
    T, Hq, H, d = 9001, 6, 3, 96
    q, k, v, da = normal((Hq, T, d), 1), normal((H, T, d), 2), normal((H, T, 128), 3), normal((T, Hq * 128), 4)
    C = torch.tensor([0, 3, 3, 5000, 8990], dtype=torch.int32, device=DEV)
    want = {}
    for window in (None, 700):
        a, lse = qk.attention_forward(q, k, v, C, window, 4)
        want[window] = (a, lse, qk.attention_backward(da, q, k, v, a, lse, C, window, 4))
    ws = qk.new_attention_workspace(T, Hq)
    graphs = {}
    for window, (a, lse, g) in want.items():   # two graphs, one workspace, replayed in turn
        outs = torch.empty_like(a), torch.empty_like(lse), {n: torch.empty_like(x) for n, x in g.items()}
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qk.attention_forward(q, k, v, C, window, 4, ws=ws, out=outs[:2])
            qk.attention_backward(da, q, k, v, *outs[:2], C, window, 4, ws=ws, out=outs[2])
        graphs[window] = graph, outs
    for _ in range(3):
        for graph, _ in graphs.values():
            graph.replay()
    torch.cuda.synchronize()
    for window, (a, lse, g) in want.items():
        oa, ol, og = graphs[window][1]
        assert torch.equal(a, oa) and torch.equal(lse, ol) and all(torch.equal(g[n], og[n]) for n in g)
    assert qk.poll_device_status(ws) == (qk.OK, 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_mixed_with_the_cache_on_a_kept_workspace(qk, fp8):
    """Calls without ``ws`` share their stream's; what one leaves there is nothing to another."""
    Hq, H, d, T, cu = 6, 6, 96, 6000, [0, 2500, 6000]
    N = (Hq + H) * d + H * 128
    y, da = normal((T, N), 1), normal((T, Hq * 128), 2)
    C, table = torch.tensor(cu, dtype=torch.int32, device=DEV), qk.build_rope_table(6000, d).to(DEV)
    pos = torch.cat([torch.arange(2500), torch.arange(3500)]).to(torch.int32).to(DEV)
    gain = torch.linspace(0.5, 1.5, d, device=DEV)
    step = normal((Hq, 2, d), 3)

    def run(own):
        ws = (lambda f: f()) if own else (lambda f: None)
        cache = qk.new_cache(2, 3600, H, d, fp8=fp8)
        norm = ws(qk.new_norm_rope_workspace)
        att = ws(lambda: qk.new_attention_workspace(T, Hq))
        c = ws(lambda: qk.new_cache_workspace(cache, Hq=Hq, budget=1000))
        q, k, v, rstd = qk.norm_rope_forward(y, pos, table, Hq, H, d, gain, gain, ws=norm)
        a, lse = qk.attention_forward(q, k, v, C, 700, 4, ws=att)
        qk.cache_append(cache, k, v, pos, cu=C, ws=c)
        out = [a, lse, *qk.decode_attention(step, cache, accumulate=True, window=700, sinks=4, ws=c)]
        g = qk.attention_backward(da, q, k, v, a, lse, C, 700, 4, ws=att)
        out += [*g.values(), *qk.decode_attention(step, cache, accumulate=True, ws=c)]
        out += qk.norm_rope_backward(*g.values(), y, rstd, pos, table, gain, gain, ws=norm).values()
        out += [qk.cache_evict(cache, 1000, 100, ws=c)]
        out += [*qk.attention_forward(q, k, v, C, ws=att), *qk.decode_attention(step, cache, accumulate=True, ws=c)]
        # (slots that no append has reached are whatever the pages' memory held: 6 x (3648 - 2500 + 3648 - 3500) of them)
        page = cache.weight.shape[2]
        live = [cache.weight[cache.table[b].long()].transpose(0, 1).reshape(H, -1)[:, :n] for b, n in ((0, 2500), (1, 3500))]
        assert page * cache.table.shape[1] == 3648
        return out + [*live, cache.lengths]
    want = run(True)
    for _ in range(2):
        assert all(torch.equal(x, o) for x, o in zip(want, run(False), strict=True))
    assert qk.poll_cache_status() == (qk.OK, 0)


def test_attention_refuses_shapes_that_the_library_does(qk):
    """What passes the binding's checks is refused by the library's."""
    for Hq, H, d, dv in ((1, 1, 0, 128), (0, 1, 96, 128), (1, 0, 96, 128), (3, 2, 96, 128), (1, 1, 80, 128)):
        q, k, v = (torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in ((Hq, 5, d), (H, 5, d), (H, 5, dv)))
        with pytest.raises(qk.QKVPError):
            qk.attention_forward(q, k, v)
        with pytest.raises(qk.QKVPError):
            qk.attention_forward(q, k, v, ws=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("d", [64, 128])
def test_windows_and_sinks_of_any_size(qk, d):
    """A window as long as the sequences, or first tokens that reach as far, hide nothing."""
    T, Hq, H = 777, 4, 2
    q, k, v, da = normal((Hq, T, d), 1), normal((H, T, d), 2), normal((H, T, 128), 3), normal((T, Hq * 128), 4)
    C = torch.tensor([0, 300, 777], dtype=torch.int32, device=DEV)

    def run(window, sinks):
        a, lse = qk.attention_forward(q, k, v, C, window, sinks)
        return a, lse, *qk.attention_backward(da, q, k, v, a, lse, C, window, sinks).values()
    want = run(None, 0)
    for window, sinks in ((477, 0), (2 ** 31 - 1, 0), (2 ** 40, 2 ** 40), (1, 477), (5, 2 ** 31 - 1), (None, 2 ** 31 - 1)):
        assert all(torch.equal(x, y) for x, y in zip(want, run(window, sinks), strict=True)), (window, sinks)
