"""Plain 64-bit forms of the paged cache's operators, on the CPU (test infrastructure only), and a
small batch builder.  Written token by token; they share no code with the package."""
from __future__ import annotations

import math

import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def rotate(x, position, rope, interleaved):
    """x [heads, D] (any type) rotated for one position, in fp64."""
    x, rot = x.double().clone(), rope.shape[1]
    c, s = rope[position, : rot // 2].double(), rope[position, rot // 2:].double()
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[:, i].clone(), x[:, j].clone()
    x[:, i], x[:, j] = a * c - b * s, b * c + a * s
    return x


def e4m3(x):
    """Nearest e4m3 value (ties to even, saturating) of non-negative fp64 x."""
    x = x.clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def quantise(x):
    """(codes 0..15 [.., D], scales fp64 [.., D / 16]) of bf16 values x [.., D]."""
    v = x.double().unflatten(-1, (-1, 16))
    s = e4m3(v.abs().amax(-1) / 6)
    y = torch.where(s[..., None] > 0, v.abs() / torch.where(s > 0, s, torch.ones_like(s))[..., None], 0.0)
    d = (y[..., None] - LEVELS).abs()
    best = d.amin(-1, keepdim=True)
    # of two equally near levels the one with the even code
    code = torch.where(d == best, torch.arange(8) + 100 * (torch.arange(8) % 2), 1000).amin(-1) % 100
    return (code + 8 * torch.signbit(v)).flatten(-2), s


def dequantise(code, s):
    v = LEVELS[(code % 8).long()] * (1 - 2 * (code // 8).double())
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def unpack(packed):
    p = packed.to(torch.int64)
    return torch.stack([p % 16, p // 16], -1).flatten(-2)


class Batch:
    """Requests with `new` tokens after `past` ones, in shuffled pages of a cache with spare pages.
    Pages that no window needs hold -1 in the table when `drop` is given as (window, sinks)."""

    def __init__(self, new, past, page, seed=0, drop=None, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.new, self.past, self.page = list(new), list(past), page
        self.lens = torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32)
        count = [-(-max(0, int(x)) // page) for x in self.lens]
        self.num_pages = sum(count) + spare
        order = torch.randperm(self.num_pages, generator=g).tolist()
        self.table = torch.full((len(count), max(1, max(count))), -1, dtype=torch.int32)
        self.seen = []
        for i, c in enumerate(count):
            for j in range(c):
                self.table[i, j] = order.pop()
            if drop is not None and drop[0]:
                w, s = drop
                lo = max(0, self.past[i] - w + 1)
                for j in range(c):
                    if (j + 1) * page <= lo and j * page >= s:
                        self.table[i, j] = -1
        self.cu = torch.zeros(len(count) + 1, dtype=torch.int32)
        self.cu[1:] = torch.cumsum(torch.tensor(self.new), 0)
        self.T = int(self.cu[-1])

    def place(self, i, j):
        return int(self.table[i, j // self.page]), j % self.page

    def on(self, device):
        return self.table.to(device), self.lens.to(device), self.cu.to(device)


def attention(q, k_of, batch, window, sinks, scale):
    """fp64 attention.  k_of(i, positions) -> (k, v) [n, kv heads, D] fp64.  Returns out, lse, the weighted
    mean of |v| per output, and the largest sum |q||k| scale per row (for error bounds)."""
    T, Hq, D = q.shape
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    big = torch.zeros(T, Hq, dtype=torch.float64)
    for i in range(len(batch.new)):
        n, length = batch.new[i], int(batch.lens[i])
        for r in range(n):
            t, pos = int(batch.cu[i]) + r, length - n + r
            if pos < 0 or length <= 0:
                continue
            j = torch.arange(pos + 1)
            if window:
                j = j[(j > pos - window) | (j < sinks)]
            k, v = k_of(i, j)
            G = Hq // k.shape[1]
            for h in range(Hq):
                x = (k[:, h // G] @ q[t, h].double()) * scale
                lse[t, h] = torch.logsumexp(x, 0)
                p = torch.exp(x - lse[t, h])
                out[t, h] = p @ v[:, h // G]
                mag[t, h] = p @ v[:, h // G].abs()
                big[t, h] = ((k[:, h // G].abs() @ q[t, h].double().abs()) * scale).max()
    return out, lse, mag, big


def bounds(out, lse, mag, big):
    """Elementwise error bounds of a bf16 output and an fp32 lse against the fp64 values.

    A score is an fp32 sum of exact products (its error is at most about D/16 roundings of partial sums,
    so 2^-20 of the sum of magnitudes is ample) and goes through an exponential of 2^-21; a weight is
    rounded to bf16 (half a step: 2^-8 of itself) before the product with the values; the output is
    rounded to bf16 once (2^-8 of itself)."""
    score = (2.0 ** -20 * big + 2.0 ** -20)[..., None]
    o = 2.0 ** -8 * out.abs() * (1 + 2.0 ** -7) + (2.0 ** -8 + 2 * score) * mag * 1.01 + 1e-30
    return o, score[..., 0] + 2.0 ** -22 * torch.where(torch.isfinite(lse), lse.abs(), 0.0)
