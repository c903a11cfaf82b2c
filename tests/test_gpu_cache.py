"""The paged cache on the GPU, through the binding, against the float64 oracle.

Bounds of the attention, fixed by the arithmetic: products of bf16 (or
de-quantised E4M3) numbers are exact in float32, so a score is off by at most
delta = (d + 8) * 2^-23 * scale * sum_j |q_j k_j| (d additions, scale and
exponent; 2^-23 a step, since a matrix unit may truncate where an addition
would round), every probability by 2 delta + 2^-20 relative (numerator, sum,
the exponential's own error), and the weights of v are rounded to bf16 (half a
step: 2^-8 relative).  So
  |a - ref|      <= 2^-8 |ref| + (2^-8 + 2 delta + 2^-20) sum_i p_i |v_i|
  |lse - ref|    <= delta + 2^-20 (1 + |ref|)
  |weight - ref| <= (2 delta + 2^-20) sum_g p_g + 2^-22 |ref|
Appended rows, codes, scales, evicted slots and moved rows are exact."""

import threading

import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def qk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_packed_reduced_gb300 import build as b
    b.build()
    import fp8_packed_reduced_gb300 as pkg
    pkg.lib()
    return pkg


def _normal(shape, seed):
    return synth._normal(shape, 1.0, seed)


def make_cache(qk, lens, H, d, page, fp8, cap=None, seed=0, spare=2):
    """A cache with random live slots.  Everything that is not live is poison:
    NaN rows, codes and scales, and page-table entries outside the pool."""
    B = len(lens)
    cap = max([cap or 1] + list(lens))
    pages = -(-cap // page)
    g = torch.Generator().manual_seed(seed)
    P = B * pages + spare
    table = torch.randperm(P, generator=g)[:B * pages].view(B, pages).to(torch.int32)
    k, v = _normal((P, H, page, d), seed + 1), _normal((P, H, page, 128), seed + 2)
    ks = vs = None
    if fp8:
        def codes(x):
            x = x.float()
            s = (x.abs().amax(-1) / torch.tensor(448.0)).clamp(min=1e-30)
            return (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s
        (k, ks), (v, vs) = codes(k), codes(v)
    weight = torch.rand((P, H, page), generator=g) ** 3
    pos = torch.randint(0, 100000, (P, H, page), generator=g, dtype=torch.int32)
    live = torch.zeros((P, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        for i in range(pages):
            live[table[b, i], :max(0, min(page, n - i * page))] = True
    dead = ~live[:, None, :].expand(P, H, page)
    for t in (ks, vs, weight):
        if t is not None:
            t[dead] = float("nan")
    pos[dead] = 2 ** 31 - 1
    for t in (k, v):
        t[dead] = 0x7F if fp8 else float("nan")
    full = table.clone()
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = (-1, 2 ** 30)[b % 2]
    to = lambda t: None if t is None else t.to(DEV).contiguous()   # noqa: E731
    cache = qk.KVCache(to(k), to(v), to(table), torch.tensor(lens, dtype=torch.int32, device=DEV), pos=to(pos),
                       weight=to(weight), k_scale=to(ks), v_scale=to(vs))
    return cache, full


def host(cache):
    c = {}
    for name in ("k", "v", "k_scale", "v_scale", "pos", "weight", "table", "lengths"):
        t = getattr(cache, name)
        c[name] = None if t is None else (synth.to_numpy_f32(t) if t.dtype == torch.bfloat16 else t.cpu().numpy()).copy()
    return c


def same(got, ref, name):
    np.testing.assert_array_equal(got, ref, err_msg=name)   # NaN equals NaN here


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------
APPEND = [  # d, page, fp8, lengths before, new rows per sequence (None: one each)
    (96, 64, False, [0, 5, 63, 64, 65], None),
    (96, 64, True, [0, 5, 63, 64, 65], None),
    (64, 16, False, [0, 1, 15, 16, 30], [17, 0, 1, 33, 2]),
    (96, 32, True, [0, 1, 31, 32, 0, 7], [0, 33, 1, 0, 64, 3]),
    (128, 128, True, [100], [157]),
    (128, 256, False, [0, 255, 256], [255, 1, 300]),
    (64, 64, True, [3] * 40, [1, 0, 2, 0, 0] * 8),
    (96, 16, False, [0, 0, 0], [0, 0, 0]),
]


@pytest.mark.parametrize("d,page,fp8,lens,new", APPEND, ids=[f"{c[0]}-{c[1]}-{'e4m3' if c[2] else 'bf16'}-B{len(c[3])}" for c in APPEND])
@pytest.mark.parametrize("in_place", [False, True])
def test_append(qk, d, page, fp8, lens, new, in_place):
    H = 3
    add = [1] * len(lens) if new is None else new
    cache, full = make_cache(qk, lens, H, d, page, fp8, cap=max(a + b for a, b in zip(lens, add)), seed=d + page)
    cache.table = full.to(DEV)
    T = sum(add)
    k, v = _normal((H, T, d), 7), _normal((H, T, 128), 8)
    if T > 2:
        k[1, 1] = 0          # a zero row: scale 1
        v[0, 2] = 1e-38      # a scale whose reciprocal overflows
    pos = torch.arange(T, dtype=torch.int32) * 3 + 1
    cu = None if new is None else torch.tensor([0] + add).cumsum(0).to(torch.int32)
    ref = host(cache)
    want = co.cache_append(ref, synth.to_numpy_f32(k), synth.to_numpy_f32(v), pos.numpy(), None if cu is None else cu.numpy())
    out = None if in_place else torch.full((len(lens),), -7, dtype=torch.int32, device=DEV)
    ws = qk.new_cache_workspace(cache, H)
    for _ in range(1 if in_place else 2):   # not in place, a second call stores the same again
        got = qk.cache_append(cache, k.to(DEV), v.to(DEV), pos.to(DEV), None if cu is None else cu.to(DEV), out, ws=ws)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    same(got.cpu().numpy(), want, "lengths")
    same(cache.lengths.cpu().numpy(), want if in_place else lens, "cache.lengths")
    have = host(cache)
    for name in ("k", "v", "k_scale", "v_scale", "pos", "weight"):
        if ref[name] is not None:
            same(have[name], ref[name], name)


def test_append_codes_of_every_mantissa(qk):
    """Every pair of a row maximum's and a value's bf16 mantissa, at scales from
    the smallest to the largest numbers: ties and near-ties of the quotient."""
    m = torch.arange(128, 256).to(torch.float32)
    vals = torch.cat([m, -m, m / 16, torch.tensor([0.0, -0.0, 1.0, -3.0] * 8)])       # 416 values a maximum
    rows = []
    for exp in (-126, -110, -80, -60, -3, 0, 40, 118):
        for top in range(128, 256, 5 if exp else 1):
            for part in vals.clamp(-top, top).view(-1, 104):
                r = torch.zeros(128)
                r[:104], r[127] = part, top
                rows.append(r.double() * 2.0 ** exp)
    v = torch.stack(rows).to(torch.bfloat16)[None]
    T = v.shape[1]
    k = v[:, :, 32:].contiguous()
    cache = qk.new_cache(1, T, 1, 96, fp8=True)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    ref = host(cache)
    co.cache_append(ref, synth.to_numpy_f32(k), synth.to_numpy_f32(v), np.zeros(T, np.int32), np.array([0, T]))
    qk.cache_append(cache, k.to(DEV), v.to(DEV), torch.zeros(T, dtype=torch.int32, device=DEV), cu)
    have = host(cache)
    slots = np.arange(T)
    for name in ("k_scale", "v_scale", "k", "v"):
        same(have[name][slots // 64, 0, slots % 64], ref[name][slots // 64, 0, slots % 64], name)


@pytest.mark.parametrize("d", [64, 96, 128])
def test_append_codes_beside_nan_and_infinity(qk, d):
    """The scale is that of the row's numbers, a NaN's code is NaN; beside an
    infinity numbers are zero."""
    k, v = _normal((1, 5, d), 1), _normal((1, 5, 128), 2)
    for x in (k, v):
        x[0, 0, 3], x[0, 0, -1] = float("nan"), -float("nan")
        x[0, 1] = float("nan")
        x[0, 2, 7] = -float("inf")
        x[0, 3, 5], x[0, 3, 6] = float("inf"), float("nan")
    cache = qk.new_cache(1, 5, 1, d, page=16, fp8=True)
    qk.cache_append(cache, k.to(DEV), v.to(DEV), torch.arange(5, dtype=torch.int32, device=DEV),
                    torch.tensor([0, 5], dtype=torch.int32, device=DEV))
    for x, pool, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        codes = pool[0, 0, :5].view(torch.float8_e4m3fn).float().cpu().numpy()
        scales, rows = scales[0, 0, :5].cpu().numpy(), synth.to_numpy_f32(x)[0]
        for t in (0, 4):
            want, s, _ = oracle.quantize(np.nan_to_num(rows[t]))
            assert scales[t] == s
            same(codes[t], np.where(np.isnan(rows[t]), np.nan, oracle.dequantize(want, 1.0)), f"row {t}")
        assert scales[1] == 1 and np.isnan(codes[1]).all()
        for t in (2, 3):
            assert scales[t] == np.inf
            same(codes[t], np.where(np.isfinite(rows[t]), 0, np.nan), f"row {t}")


def test_append_in_place_many_times(qk):
    """A decode loop: the lengths grow by one a call, on one workspace."""
    H, lens = 2, [0, 62, 7]
    cache, full = make_cache(qk, lens, H, 96, 16, False, cap=80)
    cache.table = full.to(DEV)
    ref = host(cache)
    for step in range(6):
        k, v = _normal((H, 3, 96), step), _normal((H, 3, 128), step + 50)
        pos = torch.full((3,), step, dtype=torch.int32)
        qk.cache_append(cache, k.to(DEV), v.to(DEV), pos.to(DEV))
        ref["lengths"] = co.cache_append(ref, synth.to_numpy_f32(k), synth.to_numpy_f32(v), pos.numpy())
    have = host(cache)
    for name in ("k", "v", "pos", "weight", "lengths"):
        same(have[name], ref[name], name)


def test_append_reports_what_does_not_fit(qk):
    """No room, a page outside the pool, rows outside cu: recorded, nothing
    else touched."""
    H, d = 2, 96
    cache, full = make_cache(qk, [30, 4, 0], H, d, 16, False, cap=32)
    cache.table = full.to(DEV)
    cache.table[1, 0] = cache.k.shape[0]     # one past the pool
    ws = qk.new_cache_workspace(cache, H)
    k, v, pos = _normal((H, 9, d), 1).to(DEV), _normal((H, 9, 128), 2).to(DEV), torch.arange(9, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 5, 7, 8], dtype=torch.int32, device=DEV)   # the ninth row belongs to none
    ref = host(cache)
    got = qk.cache_append(cache, k, v, pos, cu, torch.empty_like(cache.lengths), ws=ws)
    assert qk.poll_device_status(ws) == (qk.ERR_DEVICE_INPUT, 13)
    assert got.tolist() == [32, 6, 1]
    have = host(cache)
    kk, vv = synth.to_numpy_f32(k.cpu()), synth.to_numpy_f32(v.cpu())
    t0, t2 = ref["table"][0], ref["table"][2]
    for h in range(H):
        ref["k"][t0[1], h, 14:16], ref["v"][t0[1], h, 14:16] = kk[h, :2], vv[h, :2]
        ref["k"][t2[0], h, 0], ref["v"][t2[0], h, 0] = kk[h, 7], vv[h, 7]
    same(have["k"], ref["k"], "k")
    same(have["v"], ref["v"], "v")
    assert qk.poll_device_status(ws) == (qk.OK, 0)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cu,rows", [
    ([0, 2, 2, 9], [[0, 1], [], [2, 3, 4, 5]]),                # more rows than there are
    ([0, 2, 8, 20], [[0, 1], [2, 3, 4, 5], []]),
    ([1, 3, 3, 6], [[1, 2], [], [3, 4, 5]]),                   # the first row belongs to none
    ([-4, 2, 5, 6], [[0, 1], [2, 3, 4], [5]]),
    ([-9, -5, 2, 6], [[], [0, 1], [2, 3, 4, 5]]),
    ([-2 ** 31, -5, 2 ** 31 - 1, 2 ** 31 - 1], [[], [0, 1, 2, 3, 4, 5], []]),
    ([0, 5, 3, 6], [[], [], []]),                              # rows of two sequences, or of none
    ([6, 4, 2, 0], [[], [], []]),
], ids=str)
def test_append_offsets_that_do_not_fit_the_rows(qk, cu, rows, in_place):
    """Lengths grow by the rows that are stored, whatever cu says."""
    H, T, lens = 2, 6, [3, 15, 0]
    cache, full = make_cache(qk, lens, H, 96, 16, False, cap=32)
    cache.table = full.to(DEV)
    k, v, pos = _normal((H, T, 96), 1), _normal((H, T, 128), 2), torch.arange(T, dtype=torch.int32) + 50
    ref = host(cache)
    kk, vv = synth.to_numpy_f32(k), synth.to_numpy_f32(v)
    for b, mine in enumerate(rows):
        for i, t in enumerate(mine):
            at = ref["table"][b, (lens[b] + i) // 16], slice(None), (lens[b] + i) % 16
            ref["k"][at], ref["v"][at], ref["pos"][at], ref["weight"][at] = kk[:, t], vv[:, t], pos[t], 0
    ws = qk.new_cache_workspace(cache, H)
    got = qk.cache_append(cache, k.to(DEV), v.to(DEV), pos.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV),
                          None if in_place else torch.empty_like(cache.lengths), ws=ws)
    assert qk.poll_device_status(ws) == (qk.ERR_DEVICE_INPUT, 13)
    assert got.tolist() == [n + len(mine) for n, mine in zip(lens, rows)]
    have = host(cache)
    for name in ("k", "v", "pos", "weight"):
        same(have[name], ref[name], name)


def test_errors_without_a_workspace_are_polled(qk):
    """What a call without ws records can be read, also once a later call has
    needed a larger workspace; another stream has its own."""
    with torch.cuda.stream(torch.cuda.Stream()):
        assert qk.poll_cache_status() == (qk.OK, 0)
        cache, full = make_cache(qk, [32, 4], 2, 96, 16, False, cap=32)
        cache.table = full.to(DEV)
        k, v, pos = _normal((2, 2, 96), 1).to(DEV), _normal((2, 2, 128), 2).to(DEV), torch.arange(2, dtype=torch.int32, device=DEV)
        qk.cache_append(cache, k, v, pos)            # sequence 0 is full
        assert cache.lengths.tolist() == [32, 5]
        qk.decode_attention(k, cache, accumulate=True)   # a larger workspace
        assert qk.poll_cache_status(DEV) == (qk.ERR_DEVICE_INPUT, 13)
        assert qk.poll_cache_status() == (qk.OK, 0)
        qk.cache_append(cache, k, v, pos)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            assert qk.poll_cache_status() == (qk.OK, 0)
        assert qk.poll_cache_status() == (qk.ERR_DEVICE_INPUT, 13)


# ---------------------------------------------------------------------------
# Attention of one token
# ---------------------------------------------------------------------------
def check_decode(qk, cache, q, scale=None, accumulate=True, ws=None):
    H, d = cache.k.shape[1], q.shape[2]
    Hq, B, _ = q.shape
    sc = d ** -0.5 if scale is None else scale
    ref = host(cache)
    before = ref["weight"].copy()
    own = qk.new_cache_workspace(cache, Hq) if ws is None else ws
    a, lse = qk.decode_attention(q.to(DEV), cache, scale=scale, accumulate=accumulate, ws=own)
    assert qk.poll_device_status(own) == (qk.OK, 0)
    ra, rl, p, absa, size = co.decode_attention(ref, synth.to_numpy_f32(q), sc)
    a = synth.to_numpy_f32(a.cpu()).reshape(B, Hq, 128).astype(np.float64)
    lse = lse.cpu().numpy().astype(np.float64)
    delta = (d + 8) * 2.0 ** -23 * size
    bound = 2.0 ** -8 * np.abs(ra) + (2.0 ** -8 + 2 * delta[..., None] + 2.0 ** -20) * absa
    err = np.abs(a - ra)
    assert (err <= bound).all(), f"a: {np.max(err - bound)} beyond the bound at {np.argmax(err - bound)}"
    live = np.array(ref["lengths"]) > 0
    assert np.array_equal(lse[~live], rl[~live])
    assert (np.abs(lse[live] - rl[live]) <= (delta + 2.0 ** -20 * (1 + np.abs(rl)))[live]).all(), "lse"
    weight = cache.weight.cpu().numpy()
    if not accumulate:
        same(weight, before, "weight")
        return a, lse
    page, G = ref["k"].shape[2], Hq // H
    want, tol = before.astype(np.float64), np.zeros(before.shape)
    for b, n in enumerate(ref["lengths"]):
        at = ref["table"][b][np.arange(n) // page], np.arange(n) % page
        for h in range(H if n else 0):
            for g in range(h * G, (h + 1) * G):
                want[at[0], h, at[1]] += p[b][g]
                tol[at[0], h, at[1]] += (2 * delta[b, g] + 2.0 ** -20) * p[b][g]
    ok = np.isnan(want) | (np.abs(weight - want) <= tol + 2.0 ** -22 * np.abs(want))
    assert ok.all() and np.array_equal(np.isnan(weight), np.isnan(want)), "weight"
    return a, lse


SHORT = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 0, 129]
DECODE = [  # lengths, H, G, d, page, fp8
    (SHORT, 2, 1, 96, 64, False),
    (SHORT, 2, 1, 96, 16, True),
    (SHORT, 1, 8, 64, 32, False),
    (SHORT, 1, 3, 128, 128, True),
    ([1], 6, 1, 96, 64, False),
    ([0], 6, 1, 96, 64, True),
    ([1500], 2, 1, 96, 64, False),
    ([1500], 2, 1, 96, 64, True),
    ([777, 2], 2, 16, 64, 256, False),
    ([777, 2], 1, 12, 96, 16, True),
    ([300, 0, 41], 2, 9, 128, 64, False),
    ([300, 0, 41], 1, 33, 96, 64, False),
    ([2000, 3, 0, 700, 1, 1999], 5, 2, 128, 16, False),
    ([900] * 3, 16, 1, 64, 32, True),
    ([5, 900, 0, 0, 33] * 4, 3, 4, 128, 128, True),
    ([700, 0, 55], 2, 6, 128, 64, False),
    ([1200, 7], 1, 8, 96, 32, False),
    ([1200, 7], 2, 7, 96, 64, True),
    ([900, 31, 1], 1, 16, 128, 16, True),
]


@pytest.mark.parametrize("lens,H,G,d,page,fp8", DECODE,
                         ids=[f"B{len(c[0])}-max{max(c[0])}-H{c[1]}-G{c[2]}-d{c[3]}-p{c[4]}-{'e4m3' if c[5] else 'bf16'}" for c in DECODE])
def test_decode(qk, lens, H, G, d, page, fp8):
    cache, _ = make_cache(qk, lens, H, d, page, fp8, seed=len(lens) + d)
    q = _normal((H * G, len(lens), d), 5)
    check_decode(qk, cache, q, accumulate=False)
    check_decode(qk, cache, q * 3, accumulate=True)      # sharper
    check_decode(qk, cache, q, scale=0.0)                # the plain mean of v
    check_decode(qk, cache, q, scale=-0.3)


@pytest.mark.parametrize("G,d,fp8", [(1, 128, False), (1, 96, True), (16, 128, True), (8, 96, False), (2, 64, False)])
def test_decode_of_the_most_sequences(qk, G, d, fp8):
    """4096 sequences, whose list takes shared memory from the rings."""
    lens = [(i * 7) % 4 if i % 1000 else 70 + i // 100 for i in range(4096)]
    cache, _ = make_cache(qk, lens, 1, d, 16, fp8, seed=G)
    check_decode(qk, cache, _normal((G, 4096, d), 3))


@pytest.mark.parametrize("G,d,fp8", [(8, 96, False), (16, 64, False), (8, 64, True), (16, 128, True), (1, 96, False)])
def test_decode_of_a_long_sequence(qk, G, d, fp8):
    """One sequence over more than 32 blocks, whose records the last of them
    joins in more than one round (with many heads, one warp a head)."""
    cache, _ = make_cache(qk, [14001], 1, d, 64, fp8, seed=G)
    check_decode(qk, cache, _normal((G, 1, d), 4))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_large_scores(qk, fp8):
    """Scores in the thousands, of both signs, rising and falling along the
    cache: only differences to the running maximum are exponentiated."""
    lens = [400, 90]
    cache, _ = make_cache(qk, lens, 2, 96, 64, fp8, seed=3)
    check_decode(qk, cache, _normal((2, 2, 96), 6) * 256)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("size", [10, 16, 22])
@pytest.mark.parametrize("G", [1, 8, 16])
def test_decode_where_one_slot_takes_all(qk, fp8, size, G):
    """Scores so large that one probability is 1 and the others are nothing:
    a is that slot's v, however large the scores are, rounded to bf16 (2^-8),
    the probability having been rounded once (E4M3: 2^-11) and the scale's
    logarithm taken (2^-18)."""
    lens = [1, 3, 700, 1, 5000]
    cache, _ = make_cache(qk, lens, 1, 96, 32, fp8, seed=5)
    q = _normal((G, len(lens), 96), 9) * 2.0 ** size
    a, _ = qk.decode_attention(q.to(DEV), cache)
    ref, _, _, _, most = co.decode_attention(host(cache), synth.to_numpy_f32(q), 96 ** -0.5)
    one = np.zeros(most.shape, bool)      # where the best score is ahead by more than the scores may be off
    for b in range(len(lens)):
        s = synth.to_numpy_f32(q)[:, b].astype(np.float64) @ co.live_rows(host(cache), b, 0)[0].T * 96 ** -0.5
        s = np.sort(np.concatenate([s, np.full((G, 1), -np.inf)], 1), 1)
        one[b] = s[:, -1] - s[:, -2] > 25 + 4 * 104 * 2.0 ** -23 * most[b]
    assert one[[0, 3]].all() and one.mean() > 0.8
    err = np.abs(synth.to_numpy_f32(a.cpu()).reshape(ref.shape) - ref)
    bound = (2.0 ** -8 + (2.0 ** -11 + 2.0 ** -18 if fp8 else 0)) * np.abs(ref)
    assert (err <= bound)[one].all(), np.max((err / np.maximum(np.abs(ref), 1e-30))[one])


def test_decode_e4m3_rows_of_any_scale(qk):
    """k and v rows whose scales span 2^-40 .. 2^40, and a q whose values span
    2^20: what is small beside its neighbours is kept relatively."""
    cache, _ = make_cache(qk, [60, 200], 2, 96, 16, True, seed=9)
    g = torch.Generator().manual_seed(2)
    rows = cache.v_scale.shape
    cache.v_scale.mul_(torch.exp2(torch.randint(-40, 41, rows, generator=g).float()).to(DEV))
    cache.k_scale.mul_(torch.exp2(torch.randint(-12, 3, rows, generator=g).float()).to(DEV))
    q = _normal((2, 2, 96), 6)
    q[:, :, ::7] *= 2.0 ** -20
    check_decode(qk, cache, q)
    # one slot takes nearly all weight and is zero in the first half of its values
    t = cache.table.cpu()
    cache.k_scale.fill_(1 / 64)
    cache.v_scale.fill_(1.0)
    cache.k[t[0, 0], :, 3] = 0x78                       # 256 in every dim
    cache.v[t[0, 0], :, 3, :64] = 0
    check_decode(qk, cache, torch.full((2, 2, 96), 0.4, dtype=torch.bfloat16))


@pytest.mark.parametrize("G,d", [(1, 96), (2, 64), (4, 128), (5, 96), (8, 64), (9, 128), (16, 96)])
def test_decode_holds_probabilities_beyond_bf16(qk, G, d):
    """Beside the rounding of the output (half a step, 2^-8 |ref|) a bf16 cache
    adds what two bf16 leave of a probability (2^-15), what the scores' errors
    and the exponential do to it (2 delta + 2^-20), and at most 2^-23 a step
    for n additions and 32 of the joins; one bf16 would add 2^-8."""
    lens = [600, 37, 1, 250]
    cache, _ = make_cache(qk, lens, 2, d, 32, False, seed=G)
    q = _normal((2 * G, len(lens), d), 11)
    a, _ = qk.decode_attention(q.to(DEV), cache)
    ref, _, _, absa, size = co.decode_attention(host(cache), synth.to_numpy_f32(q), d ** -0.5)
    delta = (d + 8) * 2.0 ** -23 * size
    steps = (np.array(lens) + 32)[:, None] * 2.0 ** -23
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -15 + 2 * delta + 2.0 ** -20 + steps)[..., None] * absa
    err = np.abs(synth.to_numpy_f32(a.cpu()).reshape(ref.shape) - ref)
    assert (err <= bound).all(), f"{(err > bound).sum()} values, up to {np.max(err / bound)} of the bound"


@pytest.mark.parametrize("G", [1, 8])
def test_decode_infinities_in_live_values(qk, G):
    """What the formula gives: p * inf is inf for every p above zero."""
    cache, _ = make_cache(qk, [40, 3], 2, 96, 16, False)
    q = _normal((2 * G, 2, 96), 2).to(DEV)
    good = qk.decode_attention(q, cache)[0].view(2, 2 * G, 128).clone()
    t = cache.table.cpu()
    cache.v[t[0, 1], 0, 5, 7] = float("inf")
    cache.v[t[0, 2], 0, 2, 100] = float("-inf")
    cache.v[t[1, 0], 1, 1, 0] = float("inf")
    a = qk.decode_attention(q, cache)[0].view(2, 2 * G, 128)
    good[0, :G, 7], good[0, :G, 100], good[1, G:, 0] = float("inf"), -float("inf"), float("inf")
    assert torch.equal(a, good)


def test_decode_without_lse_weight_and_pos(qk):
    cache, _ = make_cache(qk, [70, 9], 2, 96, 16, False)
    q = _normal((2, 2, 96), 1).to(DEV)
    a, _ = qk.decode_attention(q, cache)
    cache.weight = cache.pos = None
    b, _ = qk.decode_attention(q, cache)
    assert torch.equal(a, b)
    with pytest.raises(ValueError, match="weight"):
        qk.decode_attention(q, cache, accumulate=True)


def test_decode_infinities_and_nan_in_live_rows(qk):
    """What the formula gives: +inf in a score or NaN anywhere in a head's live
    rows makes that head NaN and no other; a score of -inf has no weight."""
    cache, _ = make_cache(qk, [40, 40, 40], 2, 96, 16, False)
    q = torch.ones((2, 3, 96), dtype=torch.bfloat16, device=DEV)
    t = cache.table.cpu()
    good, glse = qk.decode_attention(q, cache)
    cache.k[t[0, 1], 0, 3, 5] = float("nan")
    cache.k[t[1, 2], 1, 2, 0] = float("inf")
    cache.k[t[2, 0], 0, 4, 0] = float("-inf")
    a, lse = qk.decode_attention(q, cache, accumulate=True)
    a, good = a.view(3, 2, 128).float(), good.view(3, 2, 128).float()
    assert a[0, 0].isnan().all() and a[1, 1].isnan().all()
    assert torch.equal(a[0, 1], good[0, 1]) and torch.equal(a[1, 0], good[1, 0]) and torch.equal(a[2, 1], good[2, 1])
    assert a[2, 0].isfinite().all() and lse[2, 0].isfinite()
    assert not cache.weight[t[2, 0], 0, 4].isnan()
    # every score -inf: nothing has weight, as in an empty row
    cache2, _ = make_cache(qk, [40], 2, 96, 16, False)
    cache2.k[cache2.table[0].long(), 1, :, 0] = float("-inf")
    a, lse = qk.decode_attention(q[:, :1].contiguous(), cache2)
    assert (a.view(2, 128)[1] == 0).all() and lse[0, 1] == -float("inf") and lse[0, 0].isfinite()


def test_decode_reports_bad_pages_and_lengths(qk):
    """A live page outside the pool is skipped, a length beyond the capacity
    is clamped, a negative one is empty: each is recorded."""
    cache, full = make_cache(qk, [64, 33, 16], 2, 96, 16, False, cap=64)
    cache.table = full.to(DEV)
    q = _normal((2, 3, 96), 1).to(DEV)
    ws = qk.new_cache_workspace(cache, 2)
    for page in (-1, cache.k.shape[0], 2 ** 31 - 1):
        cache.table[1, 1] = page
        w = cache.weight.clone()
        a, lse = qk.decode_attention(q, cache, accumulate=True, ws=ws)
        assert qk.poll_device_status(ws)[0] == qk.ERR_DEVICE_INPUT
        assert a.isfinite().all() and lse.isfinite().all()
        cache.weight.copy_(w)
    cache.table.copy_(full)
    good = qk.decode_attention(q, cache, ws=ws)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    for n in (65, 2 ** 31 - 1, -1):
        cache.lengths[0] = n
        a, lse = qk.decode_attention(q, cache, ws=ws)
        assert qk.poll_device_status(ws)[0] == qk.ERR_DEVICE_INPUT
        assert torch.equal(a[1:], good[0][1:])
        assert torch.equal(a[0], good[0][0]) if n > 0 else (a[0] == 0).all()


def test_decode_is_the_same_on_every_run(qk):
    lens = [3000, 5, 0, 811, 1200]
    for fp8 in (False, True):
        cache, _ = make_cache(qk, lens, 3, 96, 32, fp8)
        q = _normal((6, 5, 96), 4).to(DEV)
        w0 = cache.weight.clone()
        first = None
        for _ in range(5):
            cache.weight.copy_(w0)
            got = (*qk.decode_attention(q, cache, accumulate=True), cache.weight.nan_to_num())
            first = first or tuple(t.clone() for t in got)
            assert all(torch.equal(x, y) for x, y in zip(got, first))


def test_offsets_beyond_32_bits(qk):
    """A pool of more than 2^32 bytes in k and in v, the live pages at its end."""
    H, d, page = 8, 96, 64
    P = 50000                                     # k: 4.9 GB, v: 6.6 GB
    free, _ = torch.cuda.mem_get_info()
    if free < 30e9:
        pytest.skip("needs 30 GB of device memory")
    small, full = make_cache(qk, [150, 70], H, d, page, False)
    big = lambda t: torch.zeros((P, *t.shape[1:]), dtype=t.dtype, device=DEV)   # noqa: E731
    n = small.k.shape[0]
    cache = qk.KVCache(big(small.k), big(small.v), (full + (P - n)).to(DEV), small.lengths.clone(), pos=big(small.pos),
                       weight=big(small.weight))
    for name in ("k", "v", "pos", "weight"):
        getattr(cache, name)[P - n:] = getattr(small, name)
    small.table = full.to(DEV)
    q = _normal((H, 2, d), 3).to(DEV)
    k, v, pos = _normal((H, 2, d), 4).to(DEV), _normal((H, 2, 128), 5).to(DEV), torch.tensor([9, 8], dtype=torch.int32, device=DEV)
    for c in (small, cache):
        qk.cache_append(c, k, v, pos)
    got = [qk.decode_attention(q, c, accumulate=True) for c in (small, cache)]
    assert all(torch.equal(x, y) for x, y in zip(*got))
    slots = [qk.cache_evict(c, 65, 10) for c in (small, cache)]
    assert torch.equal(*slots)
    for name in ("k", "v", "pos", "weight"):
        same(getattr(cache, name)[P - n:].float().cpu().numpy(), getattr(small, name).float().cpu().numpy(), name)
        assert not getattr(cache, name)[:P - n].any()


# ---------------------------------------------------------------------------
# Eviction
# ---------------------------------------------------------------------------
EVICT = [  # lengths, H, d, page, fp8, budget, recent
    ([40, 0, 1, 16, 17, 100], 2, 96, 16, False, 16, 4),
    ([40, 0, 1, 16, 17, 100], 2, 96, 16, True, 16, 16),
    ([65, 64, 63, 2], 3, 64, 64, False, 1, 0),
    ([65, 64, 63, 2], 3, 128, 64, True, 1, 1),
    ([2500, 1300], 2, 96, 64, False, 1200, 300),
    ([2500, 2049], 1, 128, 256, True, 2048, 0),
    ([333] * 5, 4, 64, 32, True, 332, 17),
]


@pytest.mark.parametrize("lens,H,d,page,fp8,budget,recent", EVICT,
                         ids=[f"B{len(c[0])}-max{max(c[0])}-d{c[2]}-{'e4m3' if c[4] else 'bf16'}-{c[5]}-{c[6]}" for c in EVICT])
@pytest.mark.parametrize("values", ["distinct", "ties", "zeros", "special"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(qk, lens, H, d, page, fp8, budget, recent, values, in_place):
    cache, _ = make_cache(qk, lens, H, d, page, fp8, seed=budget)
    g = torch.Generator().manual_seed(budget + recent)
    w = cache.weight.cpu()
    live = ~w.isnan()
    if values == "ties":
        w = torch.randint(0, 4, w.shape, generator=g).float()
    elif values == "zeros":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.5, 0.0, -0.0)
    elif values == "special":
        pick = torch.randint(0, 7, w.shape, generator=g)
        w = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -1.0, 1e-40, 3.4e38])[pick]
    cache.weight.copy_(torch.where(live, w, torch.tensor(float("nan"))))
    # distinct positions, in an order of each head's own
    n = max(lens)
    for b, m in enumerate(lens):
        for h in range(H):
            order = torch.randperm(m, generator=g).to(torch.int32) * 2 + 3
            slot = torch.arange(m)
            cache.pos[cache.table[b].cpu()[slot // page].long(), h, slot % page] = order.to(DEV)
    ref = host(cache)
    want, lengths = co.cache_evict(ref, budget, recent) if budget <= n else (None, None)
    out = None if in_place else torch.full((len(lens),), -1, dtype=torch.int32, device=DEV)
    ws = qk.new_cache_workspace(cache, H, budget=budget)
    slots = qk.cache_evict(cache, budget, recent, lengths_out=out, ws=ws)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    same(slots.cpu().numpy(), want, "slots")
    same((cache.lengths if in_place else out).cpu().numpy(), lengths, "lengths")
    same(cache.lengths.cpu().numpy(), lengths if in_place else lens, "cache.lengths")
    have = host(cache)
    for name in ("k", "v", "k_scale", "v_scale", "pos", "weight"):
        if ref[name] is not None:
            same(have[name], ref[name], name)


@pytest.mark.parametrize("lens", [[2048, 2049, 100, 5000, 4], [100, 1536, 1537, 2100], [20000, 2047, 2048, 3000, 500]],
                         ids=["cap5000", "cap2100", "cap20000"])
def test_evict_short_and_long_in_one_call(qk, lens):
    """Sequences that one block selects from, beside others that a cluster does."""
    H, page, budget = 2, 16, 60
    cache, _ = make_cache(qk, lens, H, 96, page, False, seed=8)
    cache.weight.copy_((cache.weight * 8).round() / 8)          # ties too
    ref = host(cache)
    want, lengths = co.cache_evict(ref, budget, 7)
    ws = qk.new_cache_workspace(cache, H, budget=budget)
    slots = qk.cache_evict(cache, budget, 7, ws=ws)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    same(slots.cpu().numpy(), want, "slots")
    same(cache.lengths.cpu().numpy(), lengths, "lengths")
    have = host(cache)
    for name in ("k", "v", "pos", "weight"):
        same(have[name], ref[name], name)


def test_evict_equal_positions_and_extremes(qk):
    """Positions that repeat, and the ends of int32: "recent" is an exact
    difference, and ties among the protected go to the lowest slots."""
    cache, _ = make_cache(qk, [50, 50], 1, 96, 16, False)
    for b, vals in enumerate(([7] * 50, [-2 ** 31] * 20 + [2 ** 31 - 1] * 30)):
        slot = torch.arange(50)
        cache.pos[cache.table[b].cpu()[slot // 16].long(), 0, slot % 16] = torch.tensor(vals, dtype=torch.int32, device=DEV)
    ref = host(cache)
    want, _ = co.cache_evict(ref, 25, 3)
    slots = qk.cache_evict(cache, 25, 3)
    same(slots.cpu().numpy(), want, "slots")
    same(slots[0, 0].cpu().numpy(), np.arange(25), "the lowest of equals")


def test_evict_long_matches_sorted(qk):
    """Longer than one block's slots by far, against torch's stable sort."""
    H, n, budget, recent = 2, 70001, 30011, 500
    cache = qk.new_cache(1, n, H, 64, page=128, fp8=True)
    for t in (cache.k, cache.v):
        t.random_(0, 120)
    cache.k_scale.uniform_(), cache.v_scale.uniform_()
    cache.weight.uniform_().mul_(100).floor_()           # ties at the border
    cap = cache.table.shape[1] * 128
    cache.pos.copy_(torch.arange(cap, device=DEV).view(-1, 1, 128).expand(-1, H, 128))
    cache.lengths.fill_(n)
    k0, w0 = cache.k.clone(), cache.weight.clone()
    slots = qk.cache_evict(cache, budget, recent)
    for h in range(H):
        w = w0[:, h].reshape(-1)[:n].clone()
        w[n - recent:] = float("inf")
        keep = torch.zeros(n, dtype=torch.bool, device=DEV)
        keep[torch.sort(w, descending=True, stable=True).indices[:budget]] = True
        want = torch.arange(budget, device=DEV)
        want[~keep[:budget]] = keep.nonzero()[:, 0][keep.nonzero()[:, 0] >= budget]
        assert torch.equal(slots[0, h].long(), want)
        assert torch.equal(cache.k[:, h].reshape(cap, -1)[:budget], k0[:, h].reshape(cap, -1)[want])
    assert cache.lengths.tolist() == [budget]


@pytest.mark.parametrize("ties", [False, True])
def test_evict_more_slots_than_shared_memory_holds(qk, ties):
    """A sequence whose keys do not fit into a cluster's shared memory (360448),
    and one whose keys a block holds, against torch's stable sort."""
    lens, budget, recent, page, d = [400001, 3000], 2500, 700, 256, 64
    cap = -(-max(lens) // page) * page
    cache = qk.new_cache(2, cap, 1, d, page=page, fp8=True)
    for t in (cache.k, cache.v):
        t.random_(0, 120)
    cache.k_scale.uniform_(), cache.v_scale.uniform_()
    g = torch.Generator().manual_seed(3)
    w = torch.randperm(2 * cap, generator=g).float()              # distinct, exact in float32
    cache.weight.copy_((w % 50 if ties else w).view(cache.weight.shape))
    pos = torch.stack([torch.randperm(cap, generator=g) for _ in lens]).to(torch.int32).to(DEV)
    cache.pos.copy_(pos.view(cache.pos.shape))
    cache.lengths.copy_(torch.tensor(lens))
    flat = lambda t: t.reshape(2, cap, *t.shape[3:])              # noqa: E731   (the table is the identity)
    before = {n: flat(getattr(cache, n)).clone() for n in ("k", "v", "k_scale", "v_scale", "weight", "pos")}
    ws = qk.new_cache_workspace(cache, 1, budget=budget)
    slots = qk.cache_evict(cache, budget, recent, ws=ws)
    assert qk.poll_device_status(ws) == (qk.OK, 0) and cache.lengths.tolist() == [budget, budget]
    for b, n in enumerate(lens):
        key = before["weight"][b, :n].clone()
        key[before["pos"][b, :n] > before["pos"][b, :n].max() - recent] = float("inf")
        kept = torch.sort(key, descending=True, stable=True).indices[:budget].sort().values
        want = torch.arange(budget, device=DEV)
        stays = torch.zeros(budget, dtype=torch.bool, device=DEV)
        stays[kept[kept < budget]] = True
        want[~stays] = kept[kept >= budget]
        assert torch.equal(slots[b, 0].long(), want)
        for name, t in before.items():
            assert torch.equal(flat(getattr(cache, name))[b, :budget], t[b, want]), name


@pytest.mark.parametrize("fp8", [False, True])
def test_few_long_sequences_among_many(qk, fp8):
    """2600 sequences with room for 2048 slots each, nearly all of them short:
    the weights and the moves of the long ones take blocks several rounds."""
    B, cap, page, d = 2600, 2048, 16, 96
    lens = [i % 4 for i in range(B)]
    lens[0], lens[1300], lens[2599] = 2048, 1501, 1999
    cache, _ = make_cache(qk, [page] * (sum(lens) // page + B), 1, d, page, fp8, seed=4)   # its pages, and their poison's places
    table, first = torch.full((B, cap // page), -1, dtype=torch.int32), 0
    pages = cache.table[:, 0].cpu()
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = pages[first:first + m]
        first += m
        for name in ("k", "v", "k_scale", "v_scale", "weight"):
            if m and n % page and getattr(cache, name) is not None:
                getattr(cache, name)[table[b, m - 1], :, n % page:] = 0x7F if fp8 and name in "kv" else float("nan")
    cache.table, cache.lengths = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = qk.new_cache_workspace(cache, 2, budget=700)
    check_decode(qk, cache, _normal((2, B, d), 3), ws=ws)
    ref = host(cache)
    want, lengths = co.cache_evict(ref, 700, 9)
    slots = qk.cache_evict(cache, 700, 9, ws=ws)
    assert qk.poll_device_status(ws) == (qk.OK, 0)
    assert (slots[0, 0] >= 700).sum() > 192             # more than its blocks take in one round
    same(slots.cpu().numpy(), want, "slots")
    same(cache.lengths.cpu().numpy(), lengths, "lengths")
    have = host(cache)
    for name in ("k", "v", "k_scale", "v_scale", "pos", "weight"):
        if ref[name] is not None:
            same(have[name], ref[name], name)


def test_evict_reports_bad_pages(qk):
    cache, full = make_cache(qk, [64, 33], 2, 96, 16, False, cap=64)
    cache.table = full.to(DEV)
    cache.table[0, 1] = cache.k.shape[0]
    ws = qk.new_cache_workspace(cache, 2, budget=20)
    before = host(cache)
    slots = qk.cache_evict(cache, 20, 4, ws=ws)
    assert qk.poll_device_status(ws)[0] == qk.ERR_DEVICE_INPUT
    assert cache.lengths.tolist() == [20, 20] and int(slots.max()) < 64 and int(slots.min()) >= 0
    # the sequence with good pages is as the oracle has it
    ref = dict(before, table=before["table"][1:], lengths=before["lengths"][1:])
    want, _ = co.cache_evict(ref, 20, 4)
    same(slots[1:].cpu().numpy(), want, "slots")


# ---------------------------------------------------------------------------
# Streams, graphs, workspaces
# ---------------------------------------------------------------------------
def test_other_stream_and_graph(qk):
    """The three calls on a side stream, and replayed from a graph, give the
    bits of the same calls on the default stream."""
    lens, H, d = [100, 3, 64], 2, 96
    k, v = _normal((H, 3, d), 1).to(DEV), _normal((H, 3, 128), 2).to(DEV)
    q, pos = _normal((H, 3, d), 3).to(DEV), torch.tensor([100000] * 3, dtype=torch.int32, device=DEV)

    def step(cache, ws, out):
        qk.cache_append(cache, k, v, pos, ws=ws)
        qk.decode_attention(q, cache, accumulate=True, ws=ws, out=out[:2])
        qk.cache_evict(cache, 60, 8, ws=ws, out=out[2])

    def fresh():
        cache, full = make_cache(qk, lens, H, d, 16, False, cap=112)
        cache.table = full.to(DEV)
        out = (torch.empty((3, H * 128), dtype=torch.bfloat16, device=DEV), torch.empty((3, H), device=DEV),
               torch.empty((3, H, 60), dtype=torch.int32, device=DEV))
        return cache, qk.new_cache_workspace(cache, H, budget=60), out

    def state(cache, out):
        torch.cuda.synchronize()
        return [t.float().nan_to_num().cpu() for t in (cache.k, cache.v, cache.weight, cache.pos, cache.lengths, *out)]

    cache, ws, out = fresh()
    for _ in range(3):
        step(cache, ws, out)
    want = state(cache, out)

    cache, ws, out = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step(cache, ws, out)
    assert all(torch.equal(x, y) for x, y in zip(state(cache, out), want))

    cache, ws, out = fresh()
    step(cache, ws, out)      # outside the graph first
    cache, ws, out = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, ws, out)
        with pytest.raises(ValueError, match="workspace"):
            qk.decode_attention(q, cache)
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(state(cache, out), want))
    assert qk.poll_device_status(ws) == (qk.OK, 0)


def test_one_workspace_for_different_shapes(qk):
    """The counters are left at zero: calls of other shapes follow each other
    on one workspace."""
    caches = [make_cache(qk, lens, H, 96, 32, fp8, seed=i)[0]
              for i, (lens, H, fp8) in enumerate([([900], 1, False), ([5] * 30, 3, True), ([0, 700, 31], 2, False)])]
    ws = max((qk.new_cache_workspace(c, 4 * c.k.shape[1]) for c in caches), key=lambda t: t.numel())
    for _ in range(2):
        for c in caches:
            check_decode(qk, c, _normal((4 * c.k.shape[1], c.table.shape[0], 96), 2), ws=ws)


def test_kept_workspaces_are_released(qk):
    """300 MB of scores are not kept for the life of the process."""
    cache = qk.new_cache(4, 200000, 1)
    cache.lengths.fill_(0)
    q = _normal((96, 4, 96), 1).to(DEV)
    qk.release_cache_workspaces()
    before = torch.cuda.memory_allocated()
    qk.decode_attention(q, cache, accumulate=True)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before > 300e6
    qk.release_cache_workspaces()
    assert torch.cuda.memory_allocated() - before < 1e6
    a, _ = qk.decode_attention(q, cache)
    assert not a.any() and qk.poll_cache_status() == (qk.OK, 0)


def test_two_threads_on_one_stream(qk):
    """Attentions with weights and evictions of two threads on the default
    stream, on caches of different shapes, without workspaces of their own."""
    jobs = []
    for i, (lens, H, page, budget) in enumerate((([900, 33, 0], 2, 32, 40), ([300, 299, 301, 20, 7], 3, 16, 100))):
        cache, _ = make_cache(qk, lens, H, 96, page, False, seed=i)
        q = _normal((H, len(lens), 96), 7 + i).to(DEV)
        before = {n: getattr(cache, n).clone() for n in ("k", "v", "weight", "pos", "lengths")}

        def one(cache=cache, q=q, before=before, budget=budget):
            for n, t in before.items():
                getattr(cache, n).copy_(t)
            out = qk.decode_attention(q, cache, accumulate=True)
            return (*out, qk.cache_evict(cache, budget, 9),
                    *(getattr(cache, n).float().nan_to_num() for n in before))

        jobs.append((one, one()))
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2)

    def work(i):
        one, want = jobs[i]
        start.wait()
        for r in range(100):
            got = one()
            if not all(torch.equal(x, y) for x, y in zip(got, want)):
                wrong.append((i, r))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_workspace_of_any_order_of_calls(qk):
    """What one call leaves in the workspace must not be taken for another's
    counters: attentions of few and of many sequences whose pieces reach over
    blocks, evictions and appends, in turn on one workspace without a wait."""
    kinds = [([5000, 4000], 1, False), ([700, 650, 3] * 20, 4, True), ([3000], 2, False), ([900] * 33, 5, False),
             ([0, 1, 2500, 77], 3, True)]
    jobs = []
    for i, (lens, H, fp8) in enumerate(kinds):
        cache, full = make_cache(qk, lens, H, 64, 32, fp8, cap=max(lens) + 64, seed=i)
        cache.table = full.to(DEV)
        q = _normal((H, len(lens), 64), 40 + i).to(DEV)
        fresh = qk.new_cache_workspace(cache, H, budget=300)
        before = cache.weight.clone()
        want = [t.clone() for t in qk.decode_attention(q, cache, accumulate=True, ws=fresh)] + [cache.weight.nan_to_num()]
        cache.weight.copy_(before)
        jobs.append((cache, q, before, want, fresh.numel()))
    for ws in (torch.zeros(max(j[4] for j in jobs), dtype=torch.uint8, device=DEV), None):
        for order in ([0, 1, 2, 3, 4], [4, 3, 1, 0, 2], [1, 0, 1, 3, 0], [2, 2, 4, 1, 1]):
            got = []
            for i in order:
                cache, q, before, _, _ = jobs[i]
                got.append((i, [*qk.decode_attention(q, cache, accumulate=True, ws=ws)], cache.weight.nan_to_num()))
                cache.weight.copy_(before)
                B, H = cache.table.shape[0], cache.k.shape[1]
                copy = qk.KVCache(cache.k.clone(), cache.v.clone(), cache.table, cache.lengths.clone(), cache.pos.clone(),
                                  cache.weight.clone(), cache.k_scale, cache.v_scale)
                if cache.k_scale is None:
                    qk.cache_evict(copy, 300, 50, ws=ws)
                    qk.cache_append(copy, q[:H], _normal((H, B, 128), 1).to(DEV), copy.lengths.clone(), ws=ws)
            for i, out, weight in got:
                for x, y in zip((*out, weight), jobs[i][3]):
                    assert torch.equal(x, y), (order, i)
        if ws is not None:
            assert qk.poll_device_status(ws) == (qk.OK, 0)


def test_binding_refusals(qk):
    cache, _ = make_cache(qk, [20, 3], 2, 96, 16, False)
    q = _normal((2, 2, 96), 1).to(DEV)
    bad = [q[:, :1], q.float(), q[:, :, :64].contiguous(), q.transpose(0, 1), q[0]]
    for t in bad:
        with pytest.raises(ValueError):
            qk.decode_attention(t, cache)
    with pytest.raises(qk.QKVPError, match="UNSUPPORTED"):
        qk.decode_attention(_normal((3, 2, 96), 1).to(DEV), cache)
    with pytest.raises(qk.QKVPError):
        qk.cache_evict(cache, 10, 11)
    with pytest.raises(qk.QKVPError):
        qk.cache_evict(cache, 1000, 0)
    for name in ("k", "v", "table", "lengths", "pos", "weight"):
        good = getattr(cache, name)
        setattr(cache, name, good.double())
        with pytest.raises(ValueError):
            qk.decode_attention(q, cache)
        setattr(cache, name, good)
