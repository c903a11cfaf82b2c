"""Cases of the operators between the projections: a packed projection's rows
split, normalised and rotated, the causal attention over packed sequences with
a sliding window and first tokens that stay visible, both with their gradients,
and the attention of one new token over the paged cache under the same window.

  norm_rope_forward    y [T, N] (q, k, v of a token side by side; rows may be
                       part of wider ones) -> q [Hq, T, d], k [H, T, d] with
                       RMS norm, gain and rotation, v [H, T, 128], rstd
  norm_rope_backward   dq, dk, dv, y -> dy [T, N], the gains' gradients
  attention_forward    token i of a sequence attends to its tokens j <= i with
                       i - j < window or j < sinks: a [T, Hq * 128] (the output
                       projection's operand), lse [Hq, T]; rows behind the
                       last sequence give a = 0 and lse = -inf
  attention_backward   da -> dq, dk, dv
  decode_attention     one token a sequence over the cache's slots below sinks
                       and its last ``window`` ones

``own`` chooses between the framework's calls and their plain form.
"""

import math

import torch

own = False

D_V = 128
EPS = 1e-6
BASE = 10000.0
DEV = "cuda"

# What one drawn case may hold: scores of the plain form (sequences padded to
# the longest), operations, values of a packed projection, slots of a cache.
MOST_SCORES = 2.45e9
MOST_FLOPS = 1.3e12
MOST_VALUES = 49152 * 1920
MOST_SLOTS = 64 * 8192 * 6


def _case(name, op, **kw):
    c = dict(op=op, **kw)
    return dict(c, name=name) if name else c


def _attend(name, op, B, H, G, d, n, window, sinks, ragged, tail):
    return _case(name, op, B=B, H=H, G=G, d=d, n=n, window=window, sinks=sinks, ragged=ragged, tail=tail)


def _decode(name, B, H, G, d, n, window, sinks, page, fp8, accumulate, ragged):
    return _case(name, "decode", B=B, H=H, G=G, d=d, n=n, window=window, sinks=sinks, page=page, fp8=fp8,
                 accumulate=accumulate, ragged=ragged)


def _norm(name, op, T, H, G, d, gain, axes, pad, far):
    return _case(name, op, T=T, H=H, G=G, d=d, gain=gain, axes=axes, pad=pad, far=far)


def listed():
    return [
        # one short prompt: the smallest call, all latency
        _attend("attend one short", "attend", 1, 6, 1, 96, 67, 0, 0, False, 0),
        # six packed sequences of the training shape's length, each token over all before it
        _attend("attend prompts", "attend", 6, 6, 1, 96, 8192, 0, 0, False, 0),
        # ragged prompts under a window, four query heads to a K/V head, padding behind them
        _attend("attend window shared heads", "attend", 7, 8, 4, 128, 3001, 1024, 4, True, 50),
        # the gradient of a few short samples
        _attend("gradient short", "gradient", 5, 4, 2, 64, 133, 0, 0, True, 3),
        # the training step's: six sequences of 8192
        _attend("gradient prompts", "gradient", 6, 6, 1, 96, 8192, 0, 0, False, 0),
        # the same step with ragged documents and a window
        _attend("gradient window", "gradient", 6, 6, 1, 96, 8192, 1024, 4, True, 77),
        # one user far into a long document, of which the window is read
        _decode("decode window one", 1, 6, 1, 96, 131072, 4096, 4, 64, False, False, False),
        # a full batch of unequal conversations from codes, weights collected for the eviction
        _decode("decode window batch e4m3", 64, 6, 1, 96, 8192, 1024, 16, 128, True, True, True),
        # the new token of every sequence of a batch
        _norm("norm rope step", "norm", 64, 6, 1, 96, True, 1, 0, 131072),
        # the training shape's tokens
        _norm("norm rope prompts", "norm", 49152, 6, 1, 96, True, 1, 0, 8192),
        # a few images: three axes, shared heads, rows that are part of wider ones
        _norm("norm rope gradient images", "norm gradient", 1777, 4, 4, 64, True, 3, 128, 1024),
        # the training step's
        _norm("norm rope gradient prompts", "norm gradient", 49152, 6, 1, 96, True, 1, 0, 8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _held(c):
    return (c["B"] * c["n"] ** 2 * c["H"] * c["G"] <= MOST_SCORES and work(c)["flops"] <= MOST_FLOPS
            and c["B"] * c["n"] * (c["H"] * c["G"] + c["H"]) * (c["d"] + D_V) <= MOST_VALUES)


def draw(rng):
    op = rng.choice(("attend", "attend", "gradient", "gradient", "decode", "norm", "norm gradient"))
    H, G, d = rng.choice((1, 2, 3, 4, 6, 8)), rng.choice((1, 1, 1, 2, 3, 4, 8)), rng.choice((64, 96, 96, 128))
    if op.startswith("norm"):
        T = _log(rng, 1, MOST_VALUES // (H * G * d + H * (d + D_V)))
        return _norm("", op, min(T, 100000), H, G, d, rng.random() < 0.7, rng.choice((1, 1, 2, 3)), rng.choice((0, 0, 64, 136)),
                     _log(rng, 64, 131072))
    window, sinks = rng.choice((0, 1, _log(rng, 2, 8192), _log(rng, 16, 2048))), rng.choice((0, 0, 1, 4, 16, _log(rng, 1, 300)))
    if op == "decode":
        B = _log(rng, 1, 256)
        n = _log(rng, 1, max(40, min(131072, MOST_SLOTS // (B * H))))
        return _decode("", B, H, G, d, n, max(1, min(window, MOST_SLOTS // (B * H) // 4)), sinks, rng.choice((16, 32, 64, 128, 256)),
                       rng.random() < 0.4, rng.random() < 0.3, rng.random() < 0.7)
    c = _attend("", op, _log(rng, 1, 200), H, G, d, _log(rng, 1, 24000), window, sinks, rng.random() < 0.7,
                rng.choice((0, 0, 1, rng.randrange(200))))
    while not _held(c):
        c["n"] = c["n"] * 4 // 5
        c["B"] = max(1, c["B"] * 9 // 10)
    return c


# ---------------------------------------------------------------------------
# Sizes
# ---------------------------------------------------------------------------

def _lengths(c):
    """Lengths of the sequences, the first the longest; ragged ones are spread
    evenly below it, with empty ones and single tokens among them."""
    if not c["ragged"]:
        return [c["n"]] * c["B"]
    out = [c["n"]]
    for i in range(1, c["B"]):
        out.append(0 if i % 11 == 5 else 1 if i % 11 == 7 else 1 + int((c["n"] - 1) * ((i * 0.6180339887) % 1.0)))
    return out


def _pairs(n, window, sinks):
    """Pairs (i, j) of a sequence of n tokens that the attention sees."""
    w = window if window else n
    full = max(0, n - w)                      # tokens with a whole window
    seen = (n - full) * (n - full + 1) // 2 + full * w
    # token i sees min(sinks, i - w + 1) tokens before its window
    a = min(sinks, full)
    return seen + a * (a + 1) // 2 + (full - a) * sinks


def work(c):
    H, Hq, d = c["H"], c["H"] * c["G"], c["d"]
    if c["op"].startswith("norm"):
        T, N = c["T"], (Hq + H) * d + H * D_V
        table = min(c["far"], T) * d * 4
        if c["op"] == "norm":
            return dict(bytes=T * (4 * N + 4 * (Hq + H) + 4 * c["axes"]) + table, flops=0)
        return dict(bytes=T * (4 * N + 2 * (Hq + H) * d + 4 * (Hq + H) + 4 * c["axes"]) + table, flops=0)
    lens = _lengths(c)
    if c["op"] == "decode":
        total = sum(min(n, min(n, c["window"]) + min(c["sinks"], max(0, n - c["window"]))) for n in lens)
        row = (d + D_V) + 8 if c["fp8"] else 2 * (d + D_V)
        return dict(bytes=total * H * (row + (8 if c["accumulate"] else 0)) + Hq * c["B"] * (2 * d + 2 * D_V + 4),
                    flops=2 * total * Hq * (d + D_V))
    T, pairs = sum(lens) + c["tail"], sum(_pairs(n, c["window"], c["sinks"]) for n in lens) * Hq
    qkv = T * (Hq * d + H * (d + D_V)) * 2
    a = T * Hq * D_V * 2
    if c["op"] == "attend":
        return dict(bytes=qkv + a + T * Hq * 4, flops=2 * pairs * (d + D_V))
    return dict(bytes=2 * qkv + 2 * a + T * Hq * 4, flops=2 * pairs * (3 * d + 2 * D_V))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rms(x):
    """Rows normalised as the projection leaves q and k."""
    x = x.float()
    return (x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()).to(torch.bfloat16)


def _codes(x):
    """E4M3 codes of every row and its scale, amax / 448."""
    x = x.float()
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _angles(far, d):
    """Angles of positions below ``far``, [far, d / 2] in 64 bits."""
    w = BASE ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=DEV) / d)
    return torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * w


def _sections(c):
    """Pairs of a head's columns that each axis of the positions turns."""
    pairs = c["d"] // 2
    if c["axes"] == 1:
        return None
    first = pairs // (2 * c["axes"]) // 2 * 2
    rest = (pairs - first) // (c["axes"] - 1) // 2 * 2
    return (pairs - rest * (c["axes"] - 1),) + (rest,) * (c["axes"] - 1)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)   # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device=DEV)   # noqa: E731
    if case["op"].startswith("norm"):
        return _prepare_norm(case, g, randn, rand)
    if case["op"] == "decode":
        return _prepare_decode(case, g, randn, rand)
    lens, H, G, d = _lengths(case), case["H"], case["G"], case["d"]
    T = sum(lens) + case["tail"]
    s = dict(op=case["op"], window=case["window"] or None, sinks=case["sinks"], longest=max(lens))
    s["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    # queries of a head share a direction that one key in 16 has, too: the heavy hitters
    lead = randn(H, 1, d)
    s["q"] = _rms(randn(H * G, T, d) + 0.7 * lead.repeat_interleave(G, 0))
    s["k"] = _rms(randn(H, T, d) + lead * (rand(H, T, 1) < 1 / 16))
    s["v"] = randn(H, T, D_V)
    if case["op"] == "gradient":
        s["da"] = randn(T, H * G * D_V) * 0.01
        s["a"], s["lse"] = _plain_attend(s)   # what the step's forward has left
    return s


def _prepare_norm(case, g, randn, rand):
    T, H, Hq, d, far = case["T"], case["H"], case["H"] * case["G"], case["d"], case["far"]
    N = (Hq + H) * d + H * D_V
    y = randn(T, N + case["pad"]) * (0.5 + 2.0 * rand(T, 1)).to(torch.bfloat16)
    s = dict(op=case["op"], H=H, Hq=Hq, d=d, y=y[:, :N], q_gain=None, k_gain=None, sections=_sections(case))
    if case["gain"]:
        s["q_gain"], s["k_gain"] = 0.5 + rand(d), 0.5 + rand(d)
    t = torch.arange(T, device=DEV)
    if case["axes"] == 1:
        s["pos"] = (t % far).to(torch.int32)
    else:   # frames of a square picture
        side = min(far, 1 + math.isqrt(max(1, T // 2)))
        s["pos"] = torch.stack([t // side ** 2 % far, t // side % side, t % side][:case["axes"]]).to(torch.int32)
    # two pairs of columns an entry: their cosines, their sines
    angle = _angles(far, d).t().reshape(d // 4, 2, far)
    s["table"] = torch.stack([angle[:, 0].cos(), angle[:, 1].cos(), angle[:, 0].sin(), angle[:, 1].sin()], -1).float().contiguous()
    if case["op"] == "norm gradient":
        s["dq"], s["dk"], s["dv"] = randn(Hq, T, d) * 0.01, randn(H, T, d) * 0.01, randn(H, T, D_V) * 0.01
        yf = s["y"].float()[:, :(Hq + H) * d].reshape(T, Hq + H, d)
        s["rstd"] = (yf.square().mean(-1) + EPS).rsqrt().t().contiguous()   # the forward's
    return s


def _prepare_decode(case, g, randn, rand):
    lens = _lengths(case)
    B, H, G, d, page, fp8 = case["B"], case["H"], case["G"], case["d"], case["page"], case["fp8"]
    pages = -(-max(max(lens), 1) // page)
    P = B * pages + 1
    s = dict(op="decode", page=page, fp8=fp8, accumulate=case["accumulate"], window=case["window"], sinks=case["sinks"])
    s["table"] = torch.randperm(P, generator=g, device=DEV)[:B * pages].view(B, pages).to(torch.int32)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    lead = randn(H, 1, d)
    s["q"] = _rms(randn(H * G, B, d) + 0.7 * lead.repeat_interleave(G, 0))
    k = _rms(randn(P, H, page, d) + lead * (rand(P, H, page, 1) < 1 / 16))
    v = randn(P, H, page, D_V)
    s["k_scale"] = s["v_scale"] = None
    if fp8:
        k, s["k_scale"] = _codes(k)
        v, s["v_scale"] = _codes(v)
    s["k"], s["v"] = k, v
    s["weight"] = 10 * rand(P, H, page).pow(4)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import fp8_packed_reduced_gb300 as qk
    if s["op"] == "attend":
        a, lse = qk.attention_forward(s["q"], s["k"], s["v"], s["cu"], window=s["window"], sinks=s["sinks"])
        return dict(a=a, lse=lse)
    if s["op"] == "gradient":
        return qk.attention_backward(s["da"], s["q"], s["k"], s["v"], s["a"], s["lse"], s["cu"], window=s["window"],
                                     sinks=s["sinks"])
    if s["op"] == "decode":
        cache = qk.KVCache(s["k"], s["v"], s["table"], s["lengths"], weight=s["weight"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"])
        a, lse = qk.decode_attention(s["q"], cache, accumulate=s["accumulate"], window=s["window"], sinks=s["sinks"])
        return dict(a=a, lse=lse, weight=s["weight"]) if s["accumulate"] else dict(a=a, lse=lse)
    if s["op"] == "norm":
        q, k, v, rstd = qk.norm_rope_forward(s["y"], s["pos"], s["table"], s["Hq"], s["H"], s["d"], q_gain=s["q_gain"],
                                             k_gain=s["k_gain"], eps=EPS, sections=s["sections"])
        return dict(q=q, k=k, v=v, rstd=rstd)
    out = qk.norm_rope_backward(s["dq"], s["dk"], s["dv"], s["y"], s["rstd"], s["pos"], s["table"], q_gain=s["q_gain"],
                                k_gain=s["k_gain"], sections=s["sections"])
    return {n: x for n, x in out.items() if x is not None}


def _run_plain(s):
    if s["op"] == "attend":
        a, lse = _plain_attend(s)
        return dict(a=a, lse=lse)
    return {"gradient": _plain_gradient, "decode": _plain_decode, "norm": _plain_norm,
            "norm gradient": _plain_norm_gradient}[s["op"]](s)


def _padded(s):
    """Rows of the packed tokens as [B, longest] (rows past a sequence's end are
    some row of the tensor), which of them are tokens, and which pairs are seen."""
    cu = s["cu"].long()
    at = torch.arange(s["longest"], device=DEV)
    real = at < (cu[1:] - cu[:-1])[:, None]
    back = at[:, None] - at
    seen = back >= 0
    if s["window"]:
        seen = seen & ((back < s["window"]) | (at < s["sinks"]))
    return torch.where(real, cu[:-1, None] + at, 0), real, seen


def _probabilities(s, rows, seen):
    q, k = s["q"].float()[:, rows], s["k"].float()[:, rows]
    H, B, n, d = k.shape
    q = q.view(H, -1, B, n, d)
    x = torch.matmul(q, k.transpose(-1, -2)[:, None]).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    return q, k, p.div_(total), m + torch.log(total)


def _plain_attend(s):
    Hq, T, _ = s["q"].shape
    rows, real, seen = _padded(s)
    a = torch.zeros(T, Hq, D_V, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Hq, T), -math.inf, device=DEV)
    _, _, p, z = _probabilities(s, rows, seen)
    o = torch.matmul(p, s["v"].float()[:, None, rows]).flatten(0, 1)
    a[rows[real]] = o[:, real].transpose(0, 1).to(torch.bfloat16)
    lse[:, rows[real]] = z[..., 0].flatten(0, 1)[:, real]
    return a.view(T, Hq * D_V), lse


def _plain_gradient(s):
    Hq, T, d = s["q"].shape
    rows, real, seen = _padded(s)
    q, k, p, _ = _probabilities(s, rows, seen)
    H, G = q.shape[:2]
    v = s["v"].float()[:, rows]
    da = (s["da"].view(T, Hq, D_V).float().transpose(0, 1)[:, rows] * real[..., None]).view(H, G, *real.shape, D_V)
    dv = torch.matmul(p.transpose(-1, -2), da).sum(1)
    dp = torch.matmul(da, v.transpose(-1, -2)[:, None])
    ds = dp.sub_((dp * p).sum(-1, keepdim=True)).mul_(p).mul_(1 / math.sqrt(d))
    out = dict(dq=torch.matmul(ds, k[:, None]).flatten(0, 1), dk=torch.matmul(ds.transpose(-1, -2), q).sum(1), dv=dv)
    whole = dict(dq=torch.zeros_like(s["q"]), dk=torch.zeros_like(s["k"]), dv=torch.zeros_like(s["v"]))
    whole["dq"][:, rows[real]] = out["dq"][:, real].to(torch.bfloat16)
    whole["dk"][:, rows[real]] = out["dk"][:, real].to(torch.bfloat16)
    whole["dv"][:, rows[real]] = out["dv"][:, real].to(torch.bfloat16)
    return whole


def _plain_decode(s):
    lengths, table, page, W, S = s["lengths"].long(), s["table"].long(), s["page"], s["window"], s["sinks"]
    B, H = lengths.shape[0], s["k"].shape[1]
    first = torch.arange(S, device=DEV).expand(B, -1)
    last = lengths[:, None] - min(W, table.shape[1] * page) + torch.arange(min(W, table.shape[1] * page), device=DEV)
    slot = torch.cat([first, last], 1)
    live = torch.cat([first < lengths[:, None], last >= S], 1)   # no slot twice
    slot = torch.where(live, slot, 0)
    at, row = table.gather(1, slot // page), slot % page
    values = lambda x: (x.view(torch.float8_e4m3fn) if s["fp8"] else x)[at, :, row].float().transpose(1, 2)   # noqa: E731
    k, v = values(s["k"]), values(s["v"])   # [B, H, S + W, .]
    if s["fp8"]:
        k *= s["k_scale"][at, :, row].transpose(1, 2)[..., None]
        v *= s["v_scale"][at, :, row].transpose(1, 2)[..., None]
    Hq, _, d = s["q"].shape
    q = s["q"].float().transpose(0, 1).reshape(B, H, Hq // H, d)
    x = (torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)).masked_fill(~live[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    a = torch.matmul(p, torch.where(live[:, None, :, None], v, 0.0)).reshape(B, Hq * D_V).to(torch.bfloat16)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf).reshape(B, Hq)
    if not s["accumulate"]:
        return dict(a=a, lse=lse)
    s["weight"][at[live], :, row[live]] += p.sum(2).transpose(1, 2)[live]
    return dict(a=a, lse=lse, weight=s["weight"])


def _cos_sin(s):
    """Cosines and sines [T, 1, d / 2] of every token, from the table."""
    pairs = s["d"] // 2
    table = s["table"].permute(1, 0, 2)                          # [far, d / 4, 4]
    cos, sin = table[..., :2].reshape(-1, pairs), table[..., 2:].reshape(-1, pairs)
    if s["sections"] is None:
        at = s["pos"].long()
        return cos[at][:, None], sin[at][:, None]
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=DEV), torch.tensor(s["sections"], device=DEV))
    at = s["pos"].long()[axis].t()                               # [T, pairs]
    return cos.gather(0, at)[:, None], sin.gather(0, at)[:, None]


def _plain_norm(s):
    T, H, Hq, d = s["y"].shape[0], s["H"], s["Hq"], s["d"]
    y = s["y"].float()
    x = y[:, :(Hq + H) * d].reshape(T, Hq + H, d)
    rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    x = x * rstd
    if s["q_gain"] is not None:
        x = torch.cat([x[:, :Hq] * s["q_gain"], x[:, Hq:] * s["k_gain"]], 1)
    cos, sin = _cos_sin(s)
    lo, hi = x[..., :d // 2], x[..., d // 2:]
    x = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1).to(torch.bfloat16).transpose(0, 1)
    v = y[:, (Hq + H) * d:].reshape(T, H, D_V).to(torch.bfloat16).transpose(0, 1)
    return dict(q=x[:Hq].contiguous(), k=x[Hq:].contiguous(), v=v.contiguous(), rstd=rstd[..., 0].t().contiguous())


def _plain_norm_gradient(s):
    T, H, Hq, d = s["y"].shape[0], s["H"], s["Hq"], s["d"]
    x = s["y"].float()[:, :(Hq + H) * d].reshape(T, Hq + H, d)
    rstd = s["rstd"].t()[..., None]
    x = x * rstd
    cos, sin = _cos_sin(s)
    g = torch.cat([s["dq"], s["dk"]]).float().transpose(0, 1)
    lo, hi = g[..., :d // 2], g[..., d // 2:]
    g = torch.cat([lo * cos + hi * sin, hi * cos - lo * sin], -1)
    out = {}
    if s["q_gain"] is not None:
        out = dict(dq_gain=(g * x)[:, :Hq].sum((0, 1)), dk_gain=(g * x)[:, Hq:].sum((0, 1)))
        g = torch.cat([g[:, :Hq] * s["q_gain"], g[:, Hq:] * s["k_gain"]], 1)
    dx = rstd * (g - x * (g * x).mean(-1, keepdim=True))
    dy = torch.cat([dx.reshape(T, -1), s["dv"].float().transpose(0, 1).reshape(T, -1)], 1).to(torch.bfloat16)
    return dict(dy=dy, **out)


# ---------------------------------------------------------------------------
# The definition in 64 bits, one sequence and head after the other
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    lens, H, G, d, W, S = _lengths(case), case["H"], case["G"], case["d"], case["window"], case["sinks"]
    if 2.0 * sum(n * n for n in lens) * H * G * (3 * d + 2 * D_V) > 8e12:
        return None
    T, f64 = sum(lens) + case["tail"], dict(dtype=torch.float64, device=DEV)
    a, lse = torch.zeros(T, H * G * D_V, **f64), torch.full((H * G, T), -math.inf, **f64)
    dq, dk, dv = torch.zeros(H * G, T, d, **f64), torch.zeros(H, T, d, **f64), torch.zeros(H, T, D_V, **f64)
    start = 0
    for n in lens:
        for h in range(H * G):
            k, v = s["k"][h // G, start:start + n].double(), s["v"][h // G, start:start + n].double()
            for i0 in range(0, n, 2048):   # some tokens with all that they may see
                i1 = min(n, i0 + 2048)
                r = slice(start + i0, start + i1)
                j0 = max(0, i0 - W + 1) if W and not S else 0
                i, j = torch.arange(i0, i1, device=DEV)[:, None], torch.arange(j0, i1, device=DEV)[None]
                hidden = j > i
                if W:
                    hidden |= (i - j >= W) & (j >= S)
                q = s["q"][h, r].double()
                x = (q @ k[j0:i1].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1, keepdim=True)
                p = torch.exp(x - z)
                if case["op"] == "attend":
                    lse[h, r] = z[:, 0]
                    a[r, h * D_V:(h + 1) * D_V] = p @ v[j0:i1]
                    continue
                da = s["da"][r, h * D_V:(h + 1) * D_V].double()
                dp = da @ v[j0:i1].T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[h, r] = ds @ k[j0:i1]
                dk[h // G, start + j0:start + i1] += ds.T @ q
                dv[h // G, start + j0:start + i1] += p.T @ da
        start += n
    return dict(a=a, lse=lse) if case["op"] == "attend" else dict(dq=dq, dk=dk, dv=dv)


def _exact_decode(case, s):
    H, G, d, page, W, S = case["H"], case["G"], case["d"], case["page"], case["window"], case["sinks"]
    lens = _lengths(case)
    a = torch.zeros(len(lens), H * G * D_V, dtype=torch.float64, device=DEV)
    lse = torch.full((len(lens), H * G), -math.inf, dtype=torch.float64, device=DEV)
    weight = s["weight"].double()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        slot = torch.arange(n, device=DEV)
        slot = slot[(slot >= n - W) | (slot < S)]
        at, row = s["table"][b].long()[slot // page], slot % page
        for h in range(H):
            k, v = s["k"][at, h, row], s["v"][at, h, row]
            if s["fp8"]:
                k = k.view(torch.float8_e4m3fn).double() * s["k_scale"][at, h, row].double()[:, None]
                v = v.view(torch.float8_e4m3fn).double() * s["v_scale"][at, h, row].double()[:, None]
            x = s["q"][h * G:(h + 1) * G, b].double() @ k.double().T / math.sqrt(d)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            a[b, h * G * D_V:(h + 1) * G * D_V] = (p @ v.double()).reshape(-1)
            weight[at, h, row] += p.sum(0)
    return dict(a=a, lse=lse, weight=weight) if case["accumulate"] else dict(a=a, lse=lse)


def _exact_norm(case, s):
    T, H, Hq, d = case["T"], case["H"], case["H"] * case["G"], case["d"]
    angle = _angles(case["far"], d)
    pos = s["pos"].long().view(-1, T)
    sections = s["sections"] or (d // 2,)
    turn, at = [], 0
    for axis, n in enumerate(sections):
        turn.append(angle[pos[axis], at:at + n])
        at += n
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.cat(turn, -1))
    y = s["y"].double()
    gains = [s["q_gain"]] * Hq + [s["k_gain"]] * H

    def turned(x, by):
        z = torch.complex(x[:, :d // 2].contiguous(), x[:, d // 2:].contiguous()) * by
        return torch.cat([z.real, z.imag], -1)

    heads, rstds, dys = [], [], []
    dgain = torch.zeros(2, d, dtype=torch.float64, device=DEV)
    for h in range(Hq + H):
        x = y[:, h * d:(h + 1) * d]
        gain = 1.0 if gains[h] is None else gains[h].double()
        r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
        rstds.append(r[:, 0])
        if case["op"] == "norm":
            heads.append(turned(x * r * gain, turn))
            continue
        g = turned((s["dq"][h] if h < Hq else s["dk"][h - Hq]).double(), turn.conj())
        dgain[int(h >= Hq)] += (g * x * r).sum(0)
        g = g * gain
        dys.append(r * g - x * r ** 3 * (g * x).sum(-1, keepdim=True) / d)
    if case["op"] == "norm":
        v = [y[:, (Hq + H) * d + h * D_V:(Hq + H) * d + (h + 1) * D_V] for h in range(H)]
        return dict(q=torch.stack(heads[:Hq]), k=torch.stack(heads[Hq:]), v=torch.stack(v), rstd=torch.stack(rstds))
    out = dict(dy=torch.cat(dys + [s["dv"][h].double() for h in range(H)], 1))
    return dict(out, dq_gain=dgain[0], dk_gain=dgain[1]) if case["gain"] else out
