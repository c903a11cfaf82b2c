"""Refusals of the attention, of its form under a window over the cache, and of
the split, norm and rotation, on the CPU: the C entry points validate their
arguments before any CUDA call, and the binding checks tensors before those."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def qk():
    from fp8_packed_reduced_gb300 import build as b
    try:
        b.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    b.build()
    import fp8_packed_reduced_gb300 as pkg
    pkg.lib()
    return pkg


P, BIG = 4096, 1 << 60   # an aligned, non-null address that no call may reach
NAN, INF = float("nan"), float("inf")


def _at(qk, **kw):
    f = dict(T=100, Hq=4, H=2, d_qk=96, d_v=128, B=3, window=0, sinks=0, scale=0.1, cu=P)
    f.update(kw)
    return ctypes.byref(qk.AttentionDesc(*f.values()))


BAD = [(dict(T=-1), 1), (dict(Hq=0), 1), (dict(H=0), 1), (dict(d_qk=0), 1), (dict(d_v=0), 1), (dict(B=0), 1),
       (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=NAN), 1),
       (dict(scale=INF), 1), (dict(cu=None), 1), (dict(T=(1 << 24) + 1), 2), (dict(H=129, Hq=129), 2), (dict(Hq=1026), 2),
       (dict(Hq=5), 2), (dict(B=(1 << 20) + 1), 2), (dict(d_qk=80), 2), (dict(d_v=64), 2), (dict(cu=P + 4), 3)]


@pytest.mark.parametrize("change,code", BAD, ids=[str(c) for c, _ in BAD])
def test_attention_refuses_a_bad_description(qk, change, code):
    L, d = qk.lib(), _at(qk, **change)
    assert L.qkvp_attention_workspace_bytes(d) == 0
    assert L.qkvp_attention_forward(d, P, P, P, P, P, P, BIG, None) == code
    assert L.qkvp_attention_backward(d, P, P, P, P, P, P, P, P, P, P, BIG, None) == code


@pytest.mark.parametrize("scale,code", [(2.0 ** -64, 0), (2.0 ** -65, 2), (2.0 ** 64, 0), (2.0 ** 65, 2)])
def test_attention_refuses_scales_beyond_its_range(qk, scale, code):
    L, d = qk.lib(), _at(qk, scale=scale, T=0)
    assert (L.qkvp_attention_workspace_bytes(d) == 0) == (code != 0)
    assert L.qkvp_attention_forward(d, P, P, P, P, P, P, BIG, None) == code
    assert L.qkvp_attention_backward(d, P, P, P, P, P, P, P, P, P, P, BIG, None) == code


def test_attention_refuses_bad_pointers(qk):
    L, d = qk.lib(), _at(qk)
    n = L.qkvp_attention_workspace_bytes(d)
    assert n >= 1024 + 4 * 4 * 100
    for call, pointers in ((L.qkvp_attention_forward, 6), (L.qkvp_attention_backward, 10)):
        assert call(None, *[P] * pointers, BIG, None) == qk.ERR_INVALID_ARGUMENT
        for i in range(pointers):
            args = [P] * pointers
            args[i] = None
            assert call(d, *args, BIG, None) == qk.ERR_INVALID_ARGUMENT
            args[i] = P + 8
            assert call(d, *args, BIG, None) == qk.ERR_MISALIGNED
        assert call(d, *[P] * pointers, n - 1, None) == qk.ERR_WORKSPACE_TOO_SMALL
        # no tokens: nothing to launch
        assert call(_at(qk, T=0), *[None] * (pointers - 1), P, BIG, None) == qk.OK
        assert call(_at(qk, T=0), *[None] * pointers, BIG, None) == qk.ERR_INVALID_ARGUMENT


def test_decode_window_refusals(qk):
    from test_cache_abi import BAD as CACHE_BAD, _desc
    f, d = qk.lib().qkvp_decode_window_attention, ctypes.byref(_desc(qk))
    n = qk.lib().qkvp_decode_attention_workspace_bytes(d, 6, 1)
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        assert f(d, 6, window, sinks, 0.1, P, P, P, 0, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 9, 4, 0, 0.1, P, P, P, 0, P, n, None) == qk.ERR_UNSUPPORTED
    assert f(d, 6, 4, 0, NAN, P, P, P, 0, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 6, 4, 0, 0.1, None, P, P, 0, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 6, 4, 0, 0.1, P, P + 2, P, 0, P, n, None) == qk.ERR_MISALIGNED
    assert f(d, 6, 4, 0, 0.1, P, P, P, 1, P, n - 1, None) == qk.ERR_WORKSPACE_TOO_SMALL
    for change, code in CACHE_BAD:
        assert f(ctypes.byref(_desc(qk, **change)), 6, 4, 0, 0.1, P, P, P, 0, P, BIG, None) == code


def _norm(qk, sections=(0, 0, 0), **kw):
    f = dict(T=10, Hq=4, H=2, d_qk=96, d_v=128, axes=1, sections=(ctypes.c_int * 3)(*sections), max_pos=64, eps=1e-6,
             ldy=6 * 96 + 2 * 128, rope_table=P, pos=P, q_gain=P, k_gain=P)
    f.update(kw)
    return ctypes.byref(qk.NormRopeDesc(*f.values()))


NORM_BAD = [(dict(T=-1), 1), (dict(Hq=0), 1), (dict(H=0), 1), (dict(d_qk=0), 1), (dict(d_v=0), 1), (dict(axes=0), 1),
            (dict(max_pos=0), 1), (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1), (dict(rope_table=None), 1),
            (dict(pos=None), 1), (dict(q_gain=None), 1), (dict(k_gain=None), 1), (dict(ldy=6 * 96 + 2 * 128 - 8), 1),
            (dict(axes=2, sections=(24, 26, 0)), 1), (dict(axes=2, sections=(23, 25, 0)), 1),
            (dict(axes=2, sections=(-2, 50, 0)), 1), (dict(axes=3, sections=(16, 16, 14)), 1),
            (dict(axes=3, sections=(2 ** 30, 2 ** 30, 2 ** 30)), 1),
            (dict(T=(1 << 24) + 1), 2), (dict(H=129, Hq=129, ldy=1 << 20), 2), (dict(Hq=5), 2), (dict(axes=4), 2), (dict(d_qk=32), 2),
            (dict(d_v=96), 2), (dict(max_pos=1 << 30), 2), (dict(ldy=6 * 96 + 2 * 128 + 4), 3), (dict(rope_table=P + 4), 3),
            (dict(pos=P + 8), 3), (dict(q_gain=P + 4), 3)]


@pytest.mark.parametrize("change,code", NORM_BAD, ids=[str(c) for c, _ in NORM_BAD])
def test_norm_rope_refuses_a_bad_description(qk, change, code):
    L, d = qk.lib(), _norm(qk, **change)
    assert L.qkvp_norm_rope_workspace_bytes(d) == 0
    assert L.qkvp_norm_rope_forward(d, P, P, P, P, P, P, BIG, None) == code
    assert L.qkvp_norm_rope_backward(d, P, P, P, P, P, P, P, P, P, BIG, None) == code


def test_norm_rope_refuses_bad_pointers(qk):
    L, d = qk.lib(), _norm(qk)
    n = L.qkvp_norm_rope_workspace_bytes(d)
    assert n > 1024 >= L.qkvp_norm_rope_workspace_bytes(_norm(qk, q_gain=None, k_gain=None)) > 0
    for call, pointers, size in ((L.qkvp_norm_rope_forward, 6, 1024), (L.qkvp_norm_rope_backward, 9, n)):
        assert call(None, *[P] * pointers, BIG, None) == qk.ERR_INVALID_ARGUMENT
        for i in range(pointers):
            args = [P] * pointers
            args[i] = None
            assert call(d, *args, BIG, None) == qk.ERR_INVALID_ARGUMENT
            args[i] = P + 8
            assert call(d, *args, BIG, None) == qk.ERR_MISALIGNED
        assert call(d, *[P] * pointers, size - 1, None) == qk.ERR_WORKSPACE_TOO_SMALL
    assert L.qkvp_norm_rope_forward(_norm(qk, T=0, pos=None), *[None] * 5, P, BIG, None) == qk.OK
    assert L.qkvp_norm_rope_backward(_norm(qk, T=0, q_gain=None, k_gain=None), *[None] * 8, P, BIG, None) == qk.OK


def test_binding_refuses(qk, monkeypatch):
    """What the library would not see: types, shapes and layouts of tensors."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)   # noqa: E731
    q, k, v = z(4, 10, 96), z(2, 10, 96), z(2, 10, 128)
    with pytest.raises(ValueError, match="CUDA tensor"):
        qk.attention_forward(q, k, v)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    calls = []
    monkeypatch.setattr(qk, "_cache_call", lambda *a: calls.append(a[0]))
    cu, da, lse = z(3, dtype=torch.int32), z(10, 512), z(4, 10, dtype=torch.float32)
    good = dict(q=q, k=k, v=v, cu=cu)
    qk.attention_forward(**good)
    qk.attention_backward(da, q, k, v, da, lse, cu)
    assert calls == ["qkvp_attention_forward", "qkvp_attention_backward"]
    for name, x in (("q", z(4, 10, 96, dtype=torch.float32)), ("q", z(4, 96)), ("q", z(10, 4, 96).transpose(0, 1)),
                    ("k", z(2, 9, 96)), ("k", z(2, 10, 64)), ("k", z(10, 96)), ("v", z(2, 10, 96)), ("v", z(1, 10, 128)),
                    ("cu", z(1, dtype=torch.int32)), ("cu", z(3, dtype=torch.int64)), ("cu", z(3, 1, dtype=torch.int32)), ("window", 0),
                    ("window", -3), ("sinks", -1), ("out", (z(10, 511), lse)), ("out", (da, z(10, 4, dtype=torch.float32)))):
        with pytest.raises(ValueError):
            qk.attention_forward(**{**good, name: x})
    for i, x in ((0, z(10, 256)), (4, z(4, 10, 128)), (5, z(4, 10))):
        args = [da, q, k, v, da, lse]
        args[i] = x
        with pytest.raises(ValueError):
            qk.attention_backward(*args)
    with pytest.raises(ValueError, match="dq must"):
        qk.attention_backward(da, q, k, v, da, lse, out=dict(dq=k, dk=k, dv=v))
    cache = qk.new_cache(2, 100, 6, device="cpu")
    for window, sinks in ((0, 0), (-1, 0), (5, -1)):
        with pytest.raises(ValueError):
            qk.decode_attention(z(6, 2, 96), cache, window=window, sinks=sinks)

    y, pos, table, gain = z(10, 6 * 96 + 256), z(10, dtype=torch.int32), z(24, 50, 4, dtype=torch.float32), z(96, dtype=torch.float32)
    good = dict(y=y, pos=pos, rope_table=table, Hq=4, H=2, d_qk=96, q_gain=gain, k_gain=gain)
    q, k, v, rstd = qk.norm_rope_forward(**good)
    qk.norm_rope_forward(**{**good, "y": z(10, 900)[:, 4:836]})
    qk.norm_rope_forward(**{**good, "pos": z(3, 10, dtype=torch.int32), "sections": (8, 20, 20)})
    qk.norm_rope_backward(q, k, v, y, rstd, pos, table, gain, gain)
    for name, x in (("y", y.float()), ("y", z(10, 832 - 1)), ("y", z(832, 10).t()), ("y", z(1, 832).expand(10, 832)), ("pos", z(9, dtype=torch.int32)),
                    ("pos", z(10, dtype=torch.int64)), ("pos", z(1, 10, dtype=torch.int32)), ("rope_table", z(16, 50, 4, dtype=torch.float32)),
                    ("rope_table", z(24, 200, dtype=torch.float32)), ("q_gain", None), ("k_gain", z(96)), ("q_gain", z(64, dtype=torch.float32)),
                    ("sections", ()), ("sections", (48,) * 4), ("sections", (24, 24)), ("out", (k, k, v, rstd)), ("H", 3)):
        with pytest.raises(ValueError):
            qk.norm_rope_forward(**{**good, name: x})
    for i, x in ((0, z(96)), (0, z(4, 9, 96)), (2, z(2, 10, 96)), (3, z(10, 96)), (4, z(5, 10, dtype=torch.float32))):
        args = [q, k, v, y, rstd, pos, table]
        args[i] = x
        with pytest.raises(ValueError):
            qk.norm_rope_backward(*args)


def test_every_tensor_is_on_one_device(qk, monkeypatch):
    other = []     # stands for tensors on a second GPU
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: int(any(t is o for o in other)))
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: torch.device("cuda", int(any(t is o for o in other)))))
    monkeypatch.setattr(qk, "_cache_call", lambda *a: None)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cpu")   # noqa: E731
    i32, f = torch.int32, torch.float32
    q, k, v, cu, da, a, lse = z(4, 10, 96), z(2, 10, 96), z(2, 10, 128), z(3, dtype=i32), z(10, 512), z(10, 512), z(4, 10, dtype=f)
    o = dict(dq=z(4, 10, 96), dk=z(2, 10, 96), dv=z(2, 10, 128))
    y, pos, table, qg, kg, rstd, dy = (z(10, 832), z(10, dtype=i32), z(24, 50, 4, dtype=f), z(96, dtype=f), z(96, dtype=f),
                                       z(6, 10, dtype=f), z(10, 832))
    g = dict(dy=dy, dq_gain=z(96, dtype=f), dk_gain=z(96, dtype=f))

    def calls():
        return [lambda: qk.attention_forward(q, k, v, cu, out=(a, lse)), lambda: qk.attention_backward(da, q, k, v, a, lse, cu, out=o),
                lambda: qk.norm_rope_forward(y, pos, table, 4, 2, 96, qg, kg, out=(o["dq"], o["dk"], o["dv"], rstd)),
                lambda: qk.norm_rope_backward(o["dq"], o["dk"], o["dv"], y, rstd, pos, table, qg, kg, out=g)]
    for c in calls():
        c()
    uses = [[k, v, cu, a, lse], [da, k, v, a, lse, cu, *o.values()], [pos, table, qg, kg, *o.values(), rstd],
            [*o.values(), rstd, pos, table, qg, kg, *g.values()]]
    for c, tensors in zip(calls(), uses):
        for t in tensors:
            other[:] = [t]
            with pytest.raises(ValueError, match="must be on cuda:0"):
                c()
