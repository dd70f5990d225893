"""A small hybrid stack served with this library: three KDA layers, then one softmax-attention layer, over
and over, random weights.  Prompts are prefilled, then tokens are decoded one at a time; both kinds of layer
keep their state between calls (a pooled recurrent state, a paged key/value cache).

    python examples/hybrid_layers.py [--cache fp4] [--window 256 --sinks 4] [--steps 32]

It checks itself: the hidden states of the decoded tokens have to be those of prefilling all tokens at once,
up to the formats' rounding, and prints the largest difference and the time of a decode step.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_gated_delta_gb300 as kda  # noqa: E402

DEV = "cuda:0"
BF16 = torch.bfloat16


def norm(x):
    return torch.nn.functional.rms_norm(x, x.shape[-1:])


class KdaLayer:
    """Projections around kda.chunk_prefill / kda.recurrent_decode."""

    def __init__(self, width, heads, slots, gen):
        self.H, self.D = heads, 128
        n = heads * self.D
        self.w = torch.randn(width, 4 * n + heads, generator=gen, device=DEV, dtype=BF16) * width ** -0.5
        self.wo = torch.randn(n, width, generator=gen, device=DEV, dtype=BF16) * n ** -0.5
        self.A_log = torch.rand(heads, generator=gen, device=DEV)
        self.dt_bias = torch.zeros(heads, self.D, device=DEV)
        self.pool = torch.zeros(slots, heads, self.D, self.D, device=DEV)

    def __call__(self, x, batch):
        n = self.H * self.D
        q, k, v, g, b = (norm(x) @ self.w).split([n, n, n, n, self.H], 1)
        q, k, v = (t.reshape(-1, self.H, self.D).contiguous() for t in (q, k, v))
        g, b = g.float().reshape(-1, self.H, self.D).contiguous(), b.float().contiguous()
        common = (g, b, self.A_log, self.dt_bias)
        if batch.decode:
            o = kda.recurrent_decode(q, k, v, *common, self.pool, batch.slots)
        else:
            o = kda.chunk_prefill(q, k, v, *common, batch.cu, self.pool, batch.slots)
        return x + o.flatten(1) @ self.wo


class AttentionLayer:
    """Projections around kda.kv_append / kda.paged_attention."""

    def __init__(self, width, heads, kv_heads, pages, page, gen, cache, window, sinks):
        self.Hq, self.Hkv, self.D = heads, kv_heads, 128
        n = (heads + 2 * kv_heads) * self.D
        self.w = torch.randn(width, n, generator=gen, device=DEV, dtype=BF16) * width ** -0.5
        self.wo = torch.randn(heads * self.D, width, generator=gen, device=DEV, dtype=BF16) * (heads * self.D) ** -0.5
        self.cache = kda.kv_cache(pages, kv_heads, page, self.D, cache, DEV)
        self.window, self.sinks = window, sinks

    def __call__(self, x, batch):
        qkv = (norm(x) @ self.w).unflatten(1, (-1, self.D))
        q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], 1)           # views of one projection: no copies
        cu = None if batch.decode else batch.cu
        q = kda.kv_append(k, v, self.cache, batch.table, batch.lens, cu, q=q, rope=batch.rope)
        o = kda.paged_attention(q, self.cache, batch.table, batch.lens, cu, window=self.window, sinks=self.sinks,
                                max_new=batch.max_new, max_len=batch.max_len)
        return x + o.flatten(1) @ self.wo


class Batch:
    """What every layer needs to know of a call: new tokens per request and their places."""

    def __init__(self, new, past, table, rope, page):
        self.decode = all(n == 1 for n in new)
        self.cu = torch.tensor([0] + new, device=DEV).cumsum(0).int()
        self.lens = torch.tensor([n + p for n, p in zip(new, past)], device=DEV, dtype=torch.int32)
        self.slots = torch.arange(len(new), device=DEV, dtype=torch.int32)
        self.table, self.rope = table, rope
        self.max_new, self.max_len = max(new), max(n + p for n, p in zip(new, past))


def run(prompts=(300, 77, 512), steps=8, width=1024, groups=2, cache="bf16", window=0, sinks=0, page=64, seed=0, verbose=True):
    """Prefill, decode `steps` tokens, and prefill everything at once; returns the largest difference of the
    decoded tokens' hidden states relative to their largest magnitude."""
    total = [p + steps for p in prompts]
    per = -(-max(total) // page)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    table = torch.randperm(len(prompts) * per, generator=gen, device=DEV).int().view(len(prompts), per)
    rope = kda.rope_table(per * page, 128, device=DEV)
    layers = []
    for _ in range(groups):
        layers += [KdaLayer(width, 8, len(prompts), gen) for _ in range(3)]
        layers.append(AttentionLayer(width, 8, 2, len(prompts) * per, page, gen, cache, window, sinks))

    def forward(x, batch):
        for layer in layers:
            x = layer(x, batch)
        return x

    x = [torch.randn(n, width, generator=gen, device=DEV, dtype=BF16) for n in total]
    forward(torch.cat([t[:n] for t, n in zip(x, prompts)]), Batch(list(prompts), [0] * len(prompts), table, rope, page))
    got = []
    for i in range(steps):
        batch = Batch([1] * len(prompts), [p + i for p in prompts], table, rope, page)
        torch.cuda.synchronize()
        began = time.perf_counter()
        got.append(forward(torch.stack([t[n + i] for t, n in zip(x, prompts)]), batch))
        torch.cuda.synchronize()
        took = time.perf_counter() - began
    for layer in layers:
        if isinstance(layer, KdaLayer):
            layer.pool.zero_()
    whole = forward(torch.cat(x), Batch(total, [0] * len(total), table, rope, page)).split(total)
    want = torch.stack([w[n:] for w, n in zip(whole, prompts)]).float()
    got = torch.stack(got, 1).float()
    if kda.check_device_errors() != 0:
        raise RuntimeError("device error recorded")
    diff = float((got - want).abs().max() / want.abs().max())
    if verbose:
        print(f"{len(layers)} layers, {len(prompts)} requests, {cache} cache: decode step {took * 1e3:.2f} ms, "
              f"decoded against prefilled: largest difference {diff:.1e} of the largest value")
    return diff


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=("bf16", "fp4"), default="bf16")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    run(steps=a.steps, cache=a.cache, window=a.window, sinks=a.sinks)
