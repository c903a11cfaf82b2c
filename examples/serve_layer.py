"""One attention layer answering token after token: the packed projection, the
paged cache, the attention over it, the output projection and the eviction.

    python examples/serve_layer.py [--tokens 64] [--budget 96] [--fp8]

Prompts go through the projection in one call and into the cache; then every
step projects one new token per sequence, appends its k and v, attends to
everything that is cached and projects the heads' outputs back.  A sequence
that outgrows the budget keeps its latest tokens and those that the attention
has looked at most.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_packed_reduced_gb300 as qk  # noqa: E402


class ServingLayer:
    """The layer's FP8 weights, its RoPE table and its cache for B sequences."""

    def __init__(self, Wq, Wk, Wv, Wo, H, B, max_tokens, d_qk=96, d_v=128, fp8=False, budget=0, recent=0):
        dev = Wq.device
        self.H, self.d_qk, self.d_v, self.budget, self.recent = H, d_qk, d_v, budget, recent
        self.bank = qk.QKVPBank([(Wq, Wk, Wv)], H, d_qk, d_v)
        self.Wo8, _, self.wo_scale = qk.quantize_weight([Wo])
        self.table = qk.build_rope_table(max_tokens, d_qk, device=dev)
        slots = min(max_tokens, budget + 64) if budget else max_tokens
        self.cache = qk.new_cache(B, slots, H, d_qk, d_v, fp8=fp8, device=dev)
        self.ws = qk.new_cache_workspace(self.cache, H, budget=budget)
        self.seen = torch.zeros(B, dtype=torch.int32, device=dev)   # tokens of every sequence so far
        self.held = 0                                               # slots of the longest, on the host

    def _project(self, x, pos):
        W8, _, s = self.bank.layer(0)
        q, k, v, _ = qk.forward(x, pos, W8, s, self.H, self.table, self.d_qk, self.d_v)
        return q, k, v

    def _make_room(self, new):
        capacity = self.cache.table.shape[1] * self.cache.k.shape[2]
        if self.budget and self.held + new > capacity:
            qk.cache_evict(self.cache, self.budget, self.recent, ws=self.ws)
            self.held = min(self.held, self.budget)
        if self.held + new > capacity:
            raise ValueError(f"{new} more tokens do not fit beside {self.held} of {capacity}")

    def prefill(self, x, lengths):
        """Prompts side by side in x [sum(lengths), D]: their k and v go into the cache."""
        dev = x.device
        cu = torch.tensor([0, *lengths], device=dev).cumsum(0).to(torch.int32)
        n = torch.tensor(lengths, device=dev)
        start = torch.repeat_interleave(cu[:-1] - self.seen, n).to(torch.int32)
        pos = torch.arange(x.shape[0], dtype=torch.int32, device=dev) - start
        self._make_room(max(lengths))
        q, k, v = self._project(x, pos)
        qk.cache_append(self.cache, k, v, pos, cu=cu, ws=self.ws)
        self.seen += n.to(torch.int32)
        self.held += max(lengths)
        return q, k, v

    def step(self, x):
        """One new token per sequence, x [B, D].  Returns (out [B, D], a [B, H * d_v], (q, k, v))."""
        self._make_room(1)
        q, k, v = self._project(x, self.seen)
        qk.cache_append(self.cache, k, v, self.seen, ws=self.ws)
        a, _ = qk.decode_attention(q, self.cache, accumulate=self.budget > 0, ws=self.ws)
        out, _, _ = qk.oproj_forward(a, self.Wo8[0], self.wo_scale)
        self.seen += 1
        self.held += 1
        return out, a, (q, k, v)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--budget", type=int, default=96)
    ap.add_argument("--fp8", action="store_true", help="hold the cache in E4M3")
    args = ap.parse_args()
    import synth
    D, H, prompts = 768, 6, [100, 37, 128]
    dev = torch.device("cuda:0")
    w = synth.forward_inputs(synth.Shape(sum(prompts), D, H), device=dev)
    Wo = synth.oproj_inputs(1, D, H * 128, device=dev)["Wo"]
    layer = ServingLayer(w["Wq"], w["Wk"], w["Wv"], Wo, H, len(prompts), 4096, fp8=args.fp8, budget=args.budget,
                         recent=args.budget // 4)
    layer.prefill(w["x"], prompts)
    x = w["x"][:len(prompts)].contiguous()
    for _ in range(args.tokens):
        x = layer.step(x)[0]
    code, where = qk.poll_device_status(layer.ws)
    print(f"status {qk.STATUS[code]}, tokens {layer.seen.tolist()}, slots {layer.cache.lengths.tolist()}, "
          f"last output rms {x.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
