"""Refusals of the cache calls, on the CPU: the C entry points validate their
arguments before any CUDA call, and the binding checks tensors before those."""

import ctypes
import threading
import time
import types

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


P = 4096   # an aligned, non-null address that no call may reach


def _desc(qk, **kw):
    f = dict(P=8, page=64, H=6, d_qk=96, d_v=128, B=2, max_pages=4, fp8=0, k=P, v=P, k_scale=0, v_scale=0, weight=P,
             pos=P, table=P, lengths=P)
    f.update(kw)
    return qk.CacheDesc(**f)


BAD = [(dict(P=0), 1), (dict(page=0), 1), (dict(H=0), 1), (dict(B=0), 1), (dict(max_pages=0), 1), (dict(fp8=2), 1),
       (dict(k=0), 1), (dict(v=0), 1), (dict(table=0), 1), (dict(lengths=0), 1), (dict(fp8=1), 1),
       (dict(fp8=1, k_scale=P), 1), (dict(page=24), 2), (dict(page=8), 2), (dict(page=512), 2), (dict(H=129), 2),
       (dict(B=4097), 2), (dict(max_pages=1 << 20), 2), (dict(P=(1 << 31) // (6 * 64) + 1), 2), (dict(d_qk=80), 2),
       (dict(d_v=64), 2), (dict(B=4096, max_pages=1 << 17), 2), (dict(k=P + 8), 3), (dict(lengths=P + 4), 3), (dict(weight=P + 4), 3), (dict(pos=P + 8), 3)]


@pytest.mark.parametrize("change,code", BAD, ids=[str(c) for c, _ in BAD])
def test_every_call_refuses_a_bad_cache(qk, change, code):
    d = ctypes.byref(_desc(qk, **change))
    L = qk.lib()
    assert L.qkvp_cache_append_workspace_bytes(d) == 0
    assert L.qkvp_decode_attention_workspace_bytes(d, 6, 1) == 0
    assert L.qkvp_cache_evict_workspace_bytes(d, 1) == 0
    assert L.qkvp_cache_append(d, 2, P, P, P, None, P, P, 1 << 40, None) == code
    assert L.qkvp_decode_attention(d, change.get("H", 6) or 6, 0.1, P, P, P, 0, P, 1 << 40, None) == code
    assert L.qkvp_cache_evict(d, 8, 4, P, P, P, 1 << 40, None) == code


def test_null_cache(qk):
    L = qk.lib()
    assert L.qkvp_cache_append(None, 2, P, P, P, None, P, P, 1 << 40, None) == qk.ERR_INVALID_ARGUMENT
    assert L.qkvp_decode_attention(None, 6, 0.1, P, P, P, 0, P, 1 << 40, None) == qk.ERR_INVALID_ARGUMENT
    assert L.qkvp_cache_evict(None, 8, 4, P, P, P, 1 << 40, None) == qk.ERR_INVALID_ARGUMENT


def test_append_refusals(qk):
    f, d = qk.lib().qkvp_cache_append, ctypes.byref(_desc(qk))
    n = qk.lib().qkvp_cache_append_workspace_bytes(d)
    assert n > 0
    assert f(d, -1, P, P, P, P, P, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 3, P, P, P, None, P, P, n, None) == qk.ERR_INVALID_ARGUMENT      # T != B without cu
    for i in range(3):                                                           # k, v, pos
        args = [P, P, P]
        args[i] = None
        assert f(d, 2, *args, None, P, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 2, P, P, P, None, P, None, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 2, P + 2, P, P, None, P, P, n, None) == qk.ERR_MISALIGNED
    assert f(d, 2, P, P, P, P + 4, P, P, n, None) == qk.ERR_MISALIGNED
    assert f(d, 2, P, P, P, None, P + 4, P, n, None) == qk.ERR_MISALIGNED
    assert f(d, (1 << 24) + 1, P, P, P, P, P, P, n, None) == qk.ERR_UNSUPPORTED
    assert f(d, 2, P, P, P, None, P, P, n - 1, None) == qk.ERR_WORKSPACE_TOO_SMALL


def test_decode_refusals(qk):
    f, d = qk.lib().qkvp_decode_attention, ctypes.byref(_desc(qk))
    n = qk.lib().qkvp_decode_attention_workspace_bytes(d, 6, 1)
    assert n > qk.lib().qkvp_decode_attention_workspace_bytes(d, 6, 0) > 0
    assert f(d, 0, 0.1, P, P, P, 0, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 9, 0.1, P, P, P, 0, P, n, None) == qk.ERR_UNSUPPORTED            # not a multiple of 6
    assert f(d, 6 * 200, 0.1, P, P, P, 0, P, 1 << 40, None) == qk.ERR_UNSUPPORTED
    assert f(d, 6, float("nan"), P, P, P, 0, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 6, float("inf"), P, P, P, 0, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 6, 0.1, None, P, P, 0, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 6, 0.1, P, None, P, 0, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 6, 0.1, P, P, P, 0, None, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(ctypes.byref(_desc(qk, weight=0)), 6, 0.1, P, P, P, 1, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 6, 0.1, P + 2, P, P, 0, P, n, None) == qk.ERR_MISALIGNED
    assert f(d, 6, 0.1, P, P, P + 4, 0, P, n, None) == qk.ERR_MISALIGNED
    assert f(d, 6, 0.1, P, P, P, 1, P, n - 1, None) == qk.ERR_WORKSPACE_TOO_SMALL


def test_evict_refusals(qk):
    f, d = qk.lib().qkvp_cache_evict, ctypes.byref(_desc(qk))
    n = qk.lib().qkvp_cache_evict_workspace_bytes(d, 100)
    assert n > 0
    assert qk.lib().qkvp_cache_evict_workspace_bytes(d, 0) == 0
    assert qk.lib().qkvp_cache_evict_workspace_bytes(d, 4 * 64 + 1) == 0
    for budget, recent in ((0, 0), (257, 0), (100, 101), (100, -1)):
        assert f(d, budget, recent, P, P, P, 1 << 40, None) == qk.ERR_INVALID_ARGUMENT
    for change in (dict(weight=0), dict(pos=0)):
        assert f(ctypes.byref(_desc(qk, **change)), 100, 4, P, P, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 100, 4, None, P, P, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 100, 4, P, P, None, n, None) == qk.ERR_INVALID_ARGUMENT
    assert f(d, 100, 4, P + 4, P, P, n, None) == qk.ERR_MISALIGNED
    assert f(d, 100, 4, P, P, P, n - 1, None) == qk.ERR_WORKSPACE_TOO_SMALL


def test_binding_refuses_tensors_off_the_gpu(qk):
    cache = qk.new_cache(2, 100, 6, device="cpu")
    assert cache.k.shape == (4, 6, 64, 96) and cache.table.shape == (2, 2)
    z = torch.zeros((6, 2, 96), dtype=torch.bfloat16)
    for call in (lambda: qk.decode_attention(z, cache), lambda: qk.cache_evict(cache, 10, 2),
                 lambda: qk.cache_append(cache, z, z, torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_packed_descriptor_is_the_struct(qk, monkeypatch):
    """The bytes that the binding packs are those of the C struct."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    for fp8 in (False, True):
        cache = qk.new_cache(3, 100, 6, page=32, fp8=fp8, device="cpu")
        raw, H, B, d, d_v, capacity = cache._packed()
        assert (H, B, d, d_v, capacity) == (6, 3, 96, 128, 128)
        s = qk.CacheDesc.from_buffer_copy(raw)
        assert ctypes.sizeof(s) == len(raw)
        assert (s.P, s.page, s.H, s.d_qk, s.d_v, s.B, s.max_pages, s.fp8) == (12, 32, 6, 96, 128, 3, 4, int(fp8))
        for name in ("k", "v", "k_scale", "v_scale", "weight", "pos", "table", "lengths"):
            t = getattr(cache, name)
            assert (getattr(s, name) or 0) == (0 if t is None else t.data_ptr()), name


@pytest.mark.parametrize("given", [False, True], ids=["kept", "given"])
def test_calls_of_two_threads_take_turns(qk, monkeypatch, given):
    """A call's kernels pass data through the workspace: no other thread's call
    may come between them (ctypes lets the other thread run)."""
    inside, met = [], []

    def entry(*args):
        met.append(len(inside))
        inside.append(args)
        time.sleep(0.02)
        inside.pop()
        return 0

    monkeypatch.setattr(qk, "_lib_handle", types.SimpleNamespace(qkvp_cache_evict=entry, qkvp_workspace_init=lambda *a: 0))
    monkeypatch.setattr(qk, "_cache_scratch", {})
    monkeypatch.setattr(qk, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 7, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(qk, "_need_cuda_at", lambda *a: None)
    monkeypatch.setattr(torch, "device", lambda *a: "cpu")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    ws = torch.empty(64, dtype=torch.uint8) if given else None
    threads = [threading.Thread(target=qk._cache_call, args=("qkvp_cache_evict", 0, ws, lambda: 64))
               for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert met == [0] * 4


def test_tensors_on_two_devices_are_refused(qk, monkeypatch):
    """Every tensor of a call lies where the cache's k does."""
    other = []     # stands for tensors on a second GPU
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: int(any(t is o for o in other)))
    monkeypatch.setattr(torch.Tensor, "device",
                        property(lambda t: torch.device("cuda", int(any(t is o for o in other)))))
    monkeypatch.setattr(qk, "_cache_call", lambda *a: None)
    cache = qk.new_cache(2, 100, 6, fp8=True, device="cpu")
    make = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cpu")   # noqa: E731
    i32, f32 = torch.int32, torch.float32
    k, v, pos, cu = make(6, 2, 96), make(6, 2, 128), make(2, dtype=i32), make(3, dtype=i32)
    n, a, lse, slots = make(2, dtype=i32), make(2, 6 * 128), make(2, 6, dtype=f32), make(2, 6, 10, dtype=i32)

    def calls():
        qk.cache_append(cache, k, v, pos, cu, n)
        qk.decode_attention(k, cache, out=(a, lse))
        qk.cache_evict(cache, 10, 2, n, out=slots)

    calls()
    for t in (cache.v, cache.table, cache.lengths, cache.pos, cache.weight, cache.k_scale, cache.v_scale, k, v, pos, cu, n,
              a, lse, slots):
        other[:] = [t]
        with pytest.raises(ValueError, match="must be on cuda:0"):
            calls()


def test_calls_run_on_the_device_of_the_cache(qk, monkeypatch):
    """Whatever the current device is: kernels are launched on that one."""
    at, seen = [0], []

    class Guard:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            at.append(self.dev)

        def __exit__(self, *e):
            at.pop()

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[-1], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 40 + i, raising=False)
    monkeypatch.setattr(qk, "_need_cuda_at", lambda *a: None)
    monkeypatch.setattr(qk, "_lib_handle", types.SimpleNamespace(qkvp_cache_evict=lambda *a: seen.append((at[-1], a)) or 0))
    ws = torch.empty(64, dtype=torch.uint8)
    for i in (0, 1):
        qk._cache_call("qkvp_cache_evict", i, ws, lambda: 64, "x")
    assert seen == [(i, ("x", ws.data_ptr(), 64, 40 + i)) for i in (0, 1)] and at == [0]
