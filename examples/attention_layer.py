"""The attention layer of a hybrid model beside its KDA layers, served end to end.

A few packed prompts go through a KDA layer's pass and an attention layer's
prefill; the attention layer's keys and values enter the 8-bit cache, in pages that are
taken from a pool on the device; tokens are then decoded one at a time over the cache,
which accumulates the attention every cached token gets; when a sequence has passed its
budget the cache is evicted into fresh pages, the old ones go back to the pool, and
decoding goes on.

    python examples/attention_layer.py --tokens 2000 --steps 32 --budget 1024
"""
import argparse
import json
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_11_gb300 as kda  # noqa: E402

D = 128


class Layer:
    """One attention layer: its cache, the pages of its sequences, their lengths, the free pages."""

    def __init__(self, N, H, Hk, longest, budget, page, cap):
        self.N, self.H, self.Hk, self.page, self.cap = N, H, Hk, page, cap
        self.width, self.kept = -(-longest // page), -(-budget // page)
        pages = N * (self.width + self.kept)
        self.cache = kda.kda_cache_alloc(pages, Hk, page)
        self.scale = D ** -0.5
        self.free = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.count = torch.full((1,), pages, dtype=torch.int32, device="cuda")
        self.table = self.empty_table()
        self.lens = torch.zeros(N, dtype=torch.int32, device="cuda")
        self.next = torch.zeros(N, dtype=torch.int32, device="cuda")  # position of the next token

    def empty_table(self):
        return torch.full((self.N, self.width), -1, dtype=torch.int32, device="cuda")

    def reserve(self, table, lens, new):
        """Pages for `new` rows of every sequence; the lengths then."""
        return kda.kda_cache_reserve(table, lens, new, self.free, self.count, self.page, new_free_count=self.count).lens

    def prefill(self, q, k, v, cu):
        out = kda.kda_attn_fwd(q, k, v, self.scale, cap=self.cap, cu_seqlens=cu)
        lens = self.reserve(self.table, self.lens, cu[1:] - cu[:-1])
        kda.kda_cache_append(self.cache, k, v, self.table, self.lens, cu_seqlens=cu)
        self.lens = lens
        self.next = self.lens.clone()
        return out

    def decode(self, q, k, v):
        lens = self.reserve(self.table, self.lens, torch.ones_like(self.lens))
        kda.kda_cache_append(self.cache, k, v, self.table, self.lens, positions=self.next)
        self.lens, self.next = lens, self.next + 1
        return kda.kda_cache_attn(self.cache, q, self.table, self.lens, self.scale, cap=self.cap, accumulate=True)

    def evict(self, budget, recent):
        old, new = self.table, self.empty_table()
        self.reserve(new, torch.zeros_like(self.lens), self.lens.clamp(max=budget))
        lens = kda.kda_cache_evict(self.cache, old, self.lens, new, budget, recent)
        kda.kda_cache_release(old, self.lens, self.free, self.count, self.page, new_free_count=self.count)
        self.table, self.lens = new, lens


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=2000, help="tokens of each prompt")
    p.add_argument("--steps", type=int, default=32, help="tokens decoded for each sequence")
    p.add_argument("--budget", type=int, default=1024)
    p.add_argument("--recent", type=int, default=128)
    p.add_argument("--sequences", type=int, default=4)
    p.add_argument("--heads", type=int, default=16)
    p.add_argument("--kv-heads", type=int, default=4)
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    N, H, Hk, T = a.sequences, a.heads, a.kv_heads, a.sequences * a.tokens
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda") * a.tokens
    layer = Layer(N, H, Hk, a.tokens + a.steps, a.budget, page=64, cap=30.0)

    # the KDA layer before it, over the same packed rows
    rows, state = kda.kda_fwd_fused(randn(T, H, D), randn(T, H, D), randn(T, H, D), randn(T, H, D), randn(T, H),
                                    D ** -0.5, -5.0, cu_seqlens=cu)
    q = rows + randn(T, H, D)
    out = layer.prefill(q, randn(T, Hk, D), randn(T, Hk, D), cu)

    # the last prompt token once more, over the cache: what the prefill gave, but for the 8-bit codes
    last = (cu[1:] - 1).long()
    again = kda.kda_cache_attn(layer.cache, q[last].contiguous(), layer.table, layer.lens, layer.scale, cap=layer.cap)
    err = (again.float() - out[last].float()).norm() / out[last].float().norm()

    finite, after = torch.isfinite(out.float()).all(), 0
    for step in range(a.steps):
        rows, state = kda.kda_decode(randn(N, H, D), randn(N, H, D), randn(N, H, D), randn(N, H, D), randn(N, H),
                                     D ** -0.5, -5.0, initial_state=state, N=N)
        o = layer.decode(rows + randn(N, H, D), randn(N, Hk, D), randn(N, Hk, D))
        finite &= torch.isfinite(o.float()).all()
        if step == a.steps // 2:
            layer.evict(a.budget, a.recent)
            after = a.steps - 1 - step
    status = kda.kda_device_status()
    if status:
        raise kda.KdaError(status, "kda_device_status")
    report = {"sequences": N, "lens": layer.lens.tolist(), "after": after, "finite": bool(finite),
              "prefill_against_cache": float(err), "free_pages": int(layer.count)}
    print(json.dumps(report))
    return report


if __name__ == "__main__":
    main()
