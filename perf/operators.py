"""Cases of the serving operators: the paged key-value cache of the packed
projection's k and v (reduced q/k head width, v of 128), the attention of one
new token over it, and the eviction from it by accumulated attention weight.

  cache_append      k, v [H, T, d] (head-major, as the forward writes them) go
                    into the pages of their sequences, as bf16 or as E4M3
                    codes with one float32 scale per row
  decode_attention  q [G * H, B, d_qk], one token a sequence, over the pages:
                    a [B, G * H * 128] (the output projection's operand), lse
                    [B, G * H]; with accumulate, every slot's weight grows by
                    its attention probabilities
  cache_evict       every head of a sequence longer than the budget keeps the
                    slots of its most recent positions and, of the others,
                    those of the highest weight (ties: the lowest slot); kept
                    slots at or above the budget move into the freed ones

``own`` chooses between the framework's calls and their plain form.
"""

import math

import numpy as np
import torch

own = False

D_V = 128
E4M3_MAX = 448.0
DEV = "cuda"

# What one drawn case may hold: slots of all sequences and heads (padded to
# the longest sequence), tokens times heads of an append, and bytes moved.
MOST_SLOTS = 64 * 8192 * 6
MOST_ROWS = 40000 * 6
MOST_BYTES = 600e6


def _decode(name, B, H, G, d, length, page, fp8, accumulate, ragged):
    c = dict(op="decode", B=B, H=H, G=G, d=d, len=length, page=page, fp8=fp8, accumulate=accumulate, ragged=ragged)
    return dict(c, name=name) if name else c


def _append(name, B, H, d, before, new, page, fp8):
    c = dict(op="append", B=B, H=H, d=d, before=before, new=new, page=page, fp8=fp8)
    return dict(c, name=name) if name else c


def _evict(name, B, H, d, length, budget, recent, page, fp8, shuffled, ragged):
    c = dict(op="evict", B=B, H=H, d=d, len=length, budget=budget, recent=recent, page=page, fp8=fp8,
             shuffled=shuffled, ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's first tokens: the shortest call, all latency
        _decode("decode one short", 1, 6, 1, 96, 130, 64, False, False, False),
        # one user, a long document: few rows, the length has to be split
        _decode("decode one long", 1, 6, 1, 96, 131072, 64, False, False, False),
        # a full batch of unequal conversations, some of them not begun
        _decode("decode batch", 64, 6, 1, 96, 8191, 64, False, False, True),
        # the same batch twice as long from codes, heavy hitters collected for the eviction
        _decode("decode batch e4m3", 48, 6, 1, 96, 8192, 128, True, True, True),
        # many short conversations in small pages
        _decode("decode many short", 256, 8, 1, 128, 333, 16, False, True, True),
        # four query heads to each K/V head
        _decode("decode shared heads", 32, 4, 4, 64, 6001, 32, False, True, True),
        # the new token of every sequence of a batch: latency again
        _append("append step", 64, 6, 96, 4097, 1, 64, False),
        # six packed prompts of the training shape's length, to codes
        _append("append prompts e4m3", 6, 6, 96, 0, 8192, 64, True),
        # ragged continuations behind what the cache holds
        _append("append ragged", 37, 8, 128, 777, 1531, 32, False),
        # a short chat trimmed to its window
        _evict("evict short", 4, 6, 96, 517, 256, 64, 64, False, False, True),
        # prompts compressed to a quarter
        _evict("evict prompts", 24, 6, 96, 8192, 2048, 512, 64, False, False, False),
        # long histories halved, after earlier evictions have mixed the slots
        _evict("evict long e4m3", 4, 6, 96, 65536, 32768, 1024, 128, True, True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _draw(rng)
    while work(c)["bytes"] > MOST_BYTES:
        c["len"] = c["len"] * 3 // 4
    return c


def _draw(rng):
    op = rng.choice(("decode", "decode", "append", "evict"))
    H = rng.choice((1, 2, 3, 5, 6, 8, 16))
    d = rng.choice((64, 96, 96, 128))
    page = rng.choice((16, 32, 64, 128, 256))
    fp8 = rng.random() < 0.4
    B = _log(rng, 1, 256)
    if op == "append":
        new = 1 if rng.random() < 0.3 else _log(rng, 2, max(2, min(32768, MOST_ROWS // (B * H))))
        return _append("", B, H, d, rng.choice((0, _log(rng, 1, max(2, 1500000 // (B * H))))), new, page, fp8)
    length = _log(rng, 1 if op == "decode" else 24, max(40, min(131072, MOST_SLOTS // (B * H))))
    if op == "decode":
        G = rng.choice((1, 1, 1, 2, 3, 4, 8))
        return _decode("", B, H, G, d, length, page, fp8, rng.random() < 0.5, rng.random() < 0.7)
    budget = max(1, int(length * rng.uniform(0.1, 0.7)))
    return _evict("", B, H, d, length, budget, int(budget * rng.uniform(0.0, 0.6)), page, fp8, rng.random() < 0.4,
                  rng.random() < 0.6)


# ---------------------------------------------------------------------------
# Sizes
# ---------------------------------------------------------------------------

def _spread(B, most, ragged):
    """Lengths of B sequences, the first the longest; ragged ones are spread
    evenly below it, with empty ones and single tokens among them."""
    if not ragged:
        return [most] * B
    out = [most]
    for i in range(1, B):
        out.append(0 if i % 11 == 5 else 1 if i % 11 == 7 else 1 + int((most - 1) * ((i * 0.6180339887) % 1.0)))
    return out


def _sizes(case):
    """(lengths in the cache, new tokens) of every sequence."""
    if case["op"] == "append":
        before = _spread(case["B"], case["before"], True) if case["before"] else [0] * case["B"]
        new = [1] * case["B"] if case["new"] == 1 else _spread(case["B"], case["new"], case["before"] > 0)
        return before, new
    return _spread(case["B"], case["len"], case["ragged"]), [0] * case["B"]


def _row_bytes(case):
    return (case["d"] + D_V) + 8 if case["fp8"] else 2 * (case["d"] + D_V)


def work(case):
    lens, new = _sizes(case)
    B, H, d = case["B"], case["H"], case["d"]
    if case["op"] == "append":
        rows = sum(new) * H
        return dict(bytes=rows * (2 * (d + D_V) + _row_bytes(case) + 8) + 4 * sum(new) + 8 * B, flops=0)
    if case["op"] == "decode":
        Hq, total = H * case["G"], sum(lens)
        return dict(bytes=total * H * (_row_bytes(case) + (8 if case["accumulate"] else 0))
                    + Hq * B * (2 * d + 2 * D_V + 4), flops=2 * total * Hq * (d + D_V))
    budget, recent, moved, keys = case["budget"], case["recent"], 0.0, 0
    for n in lens:
        if n > budget:
            keys += n
            if case["shuffled"]:
                moved += budget * (n - budget) / n
            else:   # the recent ones are the last, the others are spread evenly
                moved += min(recent, n - budget) + (budget - recent) * max(0, n - budget - recent) / (n - recent)
    return dict(bytes=H * (8 * keys + moved * 2 * (_row_bytes(case) + 8)) + 4 * B * H * budget + 8 * B, flops=0)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rms(x):
    """Rows normalised as the projection leaves q and k."""
    x = x.float()
    return (x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()).to(torch.bfloat16)


def _codes(x):
    """E4M3 codes of every row and its scale, amax / 448."""
    x = x.float()
    amax = x.abs().amax(-1)
    # a tensor as the divisor: by a number, torch multiplies with its reciprocal
    scale = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))
    codes = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    lens, new = _sizes(case)
    B, H, d, page, fp8 = case["B"], case["H"], case["d"], case["page"], case["fp8"]
    cap = max(max(a + b for a, b in zip(lens, new)), 1)
    pages = -(-cap // page)
    P = B * pages + 1
    randn = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)   # noqa: E731
    s = dict(op=case["op"], page=page, fp8=fp8)
    s["table"] = torch.randperm(P, generator=g, device=DEV)[:B * pages].view(B, pages).to(torch.int32)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    k, v = randn(P, H, page, d), randn(P, H, page, D_V)
    if case["op"] == "decode":
        Hq = H * case["G"]
        s["q"] = _rms(randn(Hq, B, d))
        # one key in 64 points the way of its sequence's query: the heavy hitters
        lead = torch.zeros(P, H, 1, d, dtype=torch.bfloat16, device=DEV)
        lead[s["table"].long()] = s["q"][::case["G"]].transpose(0, 1)[:, None, :, None, :]
        k += lead * (torch.rand(P, H, page, 1, generator=g, device=DEV) < 1 / 64)
        s["accumulate"] = case["accumulate"]
    k = _rms(k)
    s["k_scale"] = s["v_scale"] = None
    if fp8:
        k, s["k_scale"] = _codes(k)
        v, s["v_scale"] = _codes(v)
    s["k"], s["v"] = k, v
    w = torch.rand(P, H, page, generator=g, device=DEV)
    s["weight"] = 10 * w.pow(4) * (torch.rand(P, H, page, generator=g, device=DEV) > 0.1)
    s["pos"] = torch.zeros(P, H, page, dtype=torch.int32, device=DEV)
    order = torch.arange(pages * page, device=DEV).expand(B, H, -1)
    if case.get("shuffled"):   # every head has its own order of what is live
        live = order < s["lengths"][:, None, None]
        order = torch.where(live, torch.rand(order.shape, generator=g, device=DEV), 2.0).argsort(-1).argsort(-1)
    s["pos"][s["table"].long()] = order.reshape(B, H, pages, page).transpose(1, 2).to(torch.int32)
    if case["op"] == "append":
        T = sum(new)
        s["new_k"], s["new_v"] = _rms(randn(H, T, d)), randn(H, T, D_V)
        s["cu"] = None if case["new"] == 1 else torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
        at = torch.tensor([0] + new, device=DEV).cumsum(0)
        row = torch.arange(T, device=DEV)
        seq = torch.searchsorted(at, row, right=True) - 1
        s["new_pos"] = (s["lengths"][seq] + row - at[seq]).to(torch.int32)
    if case["op"] == "evict":
        s["budget"], s["recent"] = case["budget"], case["recent"]
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _values(s, name):
    """A pool as the values it holds (E4M3 codes as such)."""
    return s[name].view(torch.float8_e4m3fn) if s["fp8"] else s[name]


def _pools(s):
    out = dict(k=_values(s, "k"), v=_values(s, "v"))
    if s["fp8"]:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import fp8_packed_reduced_gb300 as qk
    weight, pos = s["weight"], s["pos"]
    if s["op"] == "evict":   # the next pass finds what this one found
        weight, pos = weight.clone(), pos.clone()
    cache = qk.KVCache(s["k"], s["v"], s["table"], s["lengths"], pos=pos, weight=weight, k_scale=s["k_scale"],
                       v_scale=s["v_scale"])
    if s["op"] == "append":
        lengths = torch.empty_like(s["lengths"])
        qk.cache_append(cache, s["new_k"], s["new_v"], s["new_pos"], cu=s["cu"], lengths_out=lengths)
        return dict(_pools(s), weight=weight, pos=pos, lengths=lengths)
    if s["op"] == "decode":
        a, lse = qk.decode_attention(s["q"], cache, accumulate=s["accumulate"])
        return dict(a=a, lse=lse, weight=weight) if s["accumulate"] else dict(a=a, lse=lse)
    lengths = torch.empty_like(s["lengths"])
    slots = qk.cache_evict(cache, s["budget"], s["recent"], lengths_out=lengths)
    return dict(_pools(s), weight=weight, pos=pos, slots=slots, lengths=lengths)


def _run_plain(s):
    return dict(append=_plain_append, decode=_plain_decode, evict=_plain_evict)[s["op"]](s)


def _plain_append(s):
    k, v, lengths, page = s["new_k"], s["new_v"], s["lengths"], s["page"]
    B, T = lengths.shape[0], k.shape[1]
    row = torch.arange(T, device=DEV)
    if s["cu"] is None:
        seq, slot, after = row, lengths.long(), lengths + 1
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu, row, right=True) - 1
        slot = lengths[seq] + row - cu[seq]
        after = lengths + (cu[1:] - cu[:-1]).to(torch.int32)
    at, row = s["table"][seq, slot // page].long(), slot % page
    if s["fp8"]:
        k, ks = _codes(k)
        v, vs = _codes(v)
        s["k_scale"][at, :, row] = ks.transpose(0, 1)
        s["v_scale"][at, :, row] = vs.transpose(0, 1)
    s["k"][at, :, row] = k.transpose(0, 1)
    s["v"][at, :, row] = v.transpose(0, 1)
    s["weight"][at, :, row] = 0.0
    s["pos"][at, :, row] = s["new_pos"][:, None]
    return dict(_pools(s), weight=s["weight"], pos=s["pos"], lengths=after)


def _gathered(s, name):
    """A pool [P, H, page, ...] as [B, H, slots, ...] in float32."""
    x = s[name][s["table"].long()].transpose(1, 2)
    x = x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])
    return (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).float()


def _plain_decode(s):
    lengths, table = s["lengths"], s["table"]
    k, v = _gathered(s, "k"), _gathered(s, "v")
    B, H, n, d = k.shape
    if s["fp8"]:
        k *= _gathered(s, "k_scale")[..., None]
        v *= _gathered(s, "v_scale")[..., None]
    Hq = s["q"].shape[0]
    q = s["q"].float().transpose(0, 1).reshape(B, H, Hq // H, d)
    live = (torch.arange(n, device=DEV) < lengths[:, None])[:, None, None, :]
    x = (torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)).masked_fill(~live, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    a = torch.matmul(p, v).reshape(B, Hq * D_V).to(torch.bfloat16)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf).reshape(B, Hq)
    if not s["accumulate"]:
        return dict(a=a, lse=lse)
    at = table.long()
    s["weight"][at] += p.sum(2).reshape(B, H, at.shape[1], -1).transpose(1, 2)
    return dict(a=a, lse=lse, weight=s["weight"])


def _plain_evict(s):
    lengths, budget, page = s["lengths"], s["budget"], s["page"]
    weight, pos, table = s["weight"].clone(), s["pos"].clone(), s["table"].long()
    B, H, n = table.shape[0], weight.shape[1], table.shape[1] * page
    slot = torch.arange(n, device=DEV).expand(B, H, n)
    w = weight[table].transpose(1, 2).reshape(B, H, n)
    at = pos[table].transpose(1, 2).reshape(B, H, n).long()
    live = slot < lengths[:, None, None]
    over = (lengths > budget)[:, None, None]
    newest = torch.where(live, at, -1).amax(-1, keepdim=True)
    # by weight from the highest, ties in slot order, then the protected
    # before the others and the live before what no token holds
    rank = torch.where(live, torch.where(at > newest - s["recent"], 0, 1), 2)
    order = torch.sort(torch.where(w.isnan(), -math.inf, w), dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, torch.sort(rank.gather(-1, order), dim=-1, stable=True).indices)
    kept = torch.zeros_like(live).scatter(-1, order[..., :budget], True) & live
    mover = torch.sort(torch.where(kept & (slot >= budget) & over, slot, n), -1).values
    hole = ((slot < budget) & ~kept & over)[..., :budget]
    into = torch.where(hole, mover.gather(-1, (hole.cumsum(-1) - 1).clamp_min(0)), slot[..., :budget])
    slots = torch.where(live[..., :budget], into, -1).to(torch.int32)
    head = torch.arange(H, device=DEV)[None, :, None]

    def flat(i):   # row of the pools, as [P * H * page, ...]
        return (table.gather(1, (i // page).reshape(B, -1)).view(i.shape) * H + head) * page + i % page

    src, dst = flat(into), flat(slot[..., :budget])
    names = ("k", "v", "k_scale", "v_scale") if s["fp8"] else ("k", "v")
    for pool in [s[x] for x in names] + [weight, pos]:
        rows = pool.view(-1, *pool.shape[3:])
        rows[dst] = rows[src]
    return dict(_pools(s), weight=weight, pos=pos, slots=slots,
                lengths=torch.where(over[:, 0, 0], budget, lengths).to(torch.int32))


# ---------------------------------------------------------------------------
# The definition in 64 bits, one sequence and head after the other
# ---------------------------------------------------------------------------

def _grid():
    """The non-negative values of E4M3, in order."""
    sub = [m / 8 * 2.0 ** -6 for m in range(8)]
    return np.array(sub + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])


def _to_grid(x):
    """Nearest value of E4M3, ties to the even code, saturating."""
    grid = torch.from_numpy(_grid()).to(x.device)
    y = x.abs().clamp(max=E4M3_MAX).contiguous()
    hi = torch.searchsorted(grid, y).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = y - grid[lo], grid[hi] - y
    pick = torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(grid[pick], x)


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _sizes(case)
    page, H, table = s["page"], case["H"], s["table"].cpu().numpy()

    def rows(b, slots):   # (pages, rows) of slots of sequence b
        slots = np.asarray(slots)
        return torch.from_numpy(table[b][slots // page].astype(np.int64)).to(DEV), torch.from_numpy(slots % page).to(DEV)

    def pool(name, h, at):
        x = s[name][at[0], h, at[1]]
        return (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).double()

    if case["op"] == "decode":
        G, d = case["G"], case["d"]
        a = torch.zeros(len(lens), H * G * D_V, dtype=torch.float64, device=DEV)
        lse = torch.full((len(lens), H * G), -math.inf, dtype=torch.float64, device=DEV)
        weight = s["weight"].double()
        for b, n in enumerate(lens):
            for h in range(H if n else 0):
                at = rows(b, np.arange(n))
                k, v = pool("k", h, at), pool("v", h, at)
                if s["fp8"]:
                    k, v = k * pool("k_scale", h, at)[:, None], v * pool("v_scale", h, at)[:, None]
                x = s["q"][h * G:(h + 1) * G, b].double() @ k.T / math.sqrt(d)
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                p = torch.softmax(x, -1)
                a[b, h * G * D_V:(h + 1) * G * D_V] = (p @ v).reshape(-1)
                weight[at[0], h, at[1]] += p.sum(0)
        return dict(a=a, lse=lse, weight=weight) if case["accumulate"] else dict(a=a, lse=lse)

    pools = {n: _values(s, n).double() for n in ("k", "v")}
    if s["fp8"]:
        pools.update(k_scale=s["k_scale"].double(), v_scale=s["v_scale"].double())
    pools.update(weight=s["weight"].double(), pos=s["pos"].clone())
    if case["op"] == "append":
        start = 0
        for b, (n, m) in enumerate(zip(lens, new)):
            if m:
                at = rows(b, np.arange(n, n + m))
                for name in ("k", "v"):
                    x = s["new_" + name][:, start:start + m].transpose(0, 1).double()
                    if s["fp8"]:
                        amax = x.abs().amax(-1)
                        scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
                        pools[name + "_scale"][at[0], :, at[1]] = scale
                        # by definition the quotient is a float32 one, by the stored scale
                        x = _to_grid((x.float() / scale.float()[..., None]).double())
                    pools[name][at[0], :, at[1]] = x
                pools["weight"][at[0], :, at[1]] = 0.0
                pools["pos"][at[0], :, at[1]] = s["new_pos"][start:start + m, None]
            start += m
        return dict(pools, lengths=torch.tensor([a + b for a, b in zip(lens, new)], dtype=torch.int32))
    budget = case["budget"]
    slots = np.full((len(lens), H, budget), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        slots[b, :, :min(n, budget)] = np.arange(min(n, budget))
        for h in range(H if n > budget else 0):
            at = rows(b, np.arange(n))
            w, p = s["weight"][at[0], h, at[1]].double().cpu().numpy(), s["pos"][at[0], h, at[1]].cpu().numpy().astype(np.int64)
            protected = p > p.max() - case["recent"]
            best = np.lexsort((np.arange(n), -w, ~protected))[:budget]
            free = np.setdiff1d(np.arange(budget), best)
            moved = np.sort(best[best >= budget])
            slots[b, h, free] = moved
            if len(free):
                src, dst = rows(b, moved), rows(b, free)
                for x in pools.values():
                    x[dst[0], h, dst[1]] = x[src[0], h, src[1]]
    return dict(pools, slots=torch.from_numpy(slots),
                lengths=torch.tensor([min(n, budget) for n in lens], dtype=torch.int32))
