"""Cases of the paged key/value cache operators: what each is called with, its plain form and its
definition in 64 bits.

Three operators serve the softmax-attention layers of a hybrid model, next to the gated delta rule
of its other layers:

  append     rotates the new tokens' queries and keys by their positions and writes keys and values
             into a paged cache, in bfloat16 or in 4 bits;
  attend     attention of the new tokens over a paged bfloat16 cache: causal, over all earlier
             tokens or over a sliding window and a few first tokens that stay visible;
  attend4    the same over a cache held in 4 bits.

A case is a batch of requests.  Request i has `new` tokens in this call, drawn from
[new_lo, new_hi], after a past of [past_lo, past_hi] tokens; both follow from `lens` alone.
Cache layout: [pages][kv heads][page tokens][channels]; token j of request i sits at row j % page of
page block_table[i][j // page].  In 4 bits two channels share a byte (the even one in its low half)
as sign, two exponent bits and one mantissa bit (0, .5, 1, 1.5, 2, 3, 4, 6), and each 16 channels
share a scale in float8 e4m3: a group's largest magnitude / 6, rounded to nearest.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _case(name, op, batch, new, past, **kw):
    c = dict(name=name, op=op, batch=batch, new_lo=new[0], new_hi=new[1], past_lo=past[0], past_hi=past[1], lens=1,
             q_heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0, rot=128, interleaved=False, bits=16)
    c.update(kw)
    return c


def listed():
    return [
        # one token of one request: a chat's decode step, where the call's own latency is all there is
        _case("append_token", "append", 1, (1, 1), (4095, 4095)),
        # eight packed prompts, the lengths of the varlen prefill workload
        _case("append_prompts", "append", 8, (512, 4096), (0, 0)),
        # a decode step of a full batch into a 4-bit cache
        _case("append4_step", "append", 256, (1, 1), (512, 4096), bits=4),
        # one long prompt of odd length, half of the channels rotated, in neighbouring pairs
        _case("append4_prompt", "append", 1, (16411, 16411), (0, 0), bits=4, rot=64, interleaved=True),
        # one token of one request over a short history: latency
        _case("attend_token", "attend", 1, (1, 1), (4095, 4095)),
        # a decode step of a batch with ragged histories
        _case("attend_step", "attend", 64, (1, 1), (511, 8191)),
        # a decode step of a full batch with a sliding window behind long histories, four sinks
        _case("attend_step_window", "attend", 256, (1, 1), (511, 16383), window=4096, sinks=4),
        # verification of four draft tokens a request
        _case("attend_verify", "attend", 64, (4, 4), (512, 4096)),
        # packed prompts with a window, page of 16
        _case("attend_prompts_window", "attend", 8, (512, 4096), (0, 0), window=1024, sinks=4, page=16),
        # the eighth 4096-token call of a long prompt that is prefilled in parts
        _case("attend_chunk", "attend", 1, (4096, 4096), (28672, 28672)),
        # a decode step over long documents held in 4 bits
        _case("attend4_long", "attend", 16, (1, 1), (4095, 131071), bits=4),
        # a part of a prompt against a 4-bit past, odd lengths
        _case("attend4_chunk", "attend", 4, (500, 1030), (2000, 9000), bits=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend"])
    bits = rng.choice([16, 4])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    rot = rng.choice([32, 64, dim])
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["step", "verify", "prompt"])
    batch = _log(rng, 1, 256) if kind != "prompt" else _log(rng, 1, 16)
    top = {"step": 1, "verify": 16, "prompt": 4500}[kind]
    hi = _log(rng, 1, top)
    past = _log(rng, 1, 60000)
    window = rng.choice([0, 0, _log(rng, 1, 8192)])
    sinks = rng.choice([0, 1, 4, 200]) if window else 0
    c = _case("", op, batch, (max(1, hi // 3), hi), (past // 4, past), lens=rng.randrange(1 << 30), q_heads=kv * group,
              kv_heads=kv, dim=dim, page=page, window=window, sinks=sinks, rot=rot, interleaved=rng.random() < 0.4, bits=bits)
    del c["name"]
    while True:  # no dearer than the largest listed ones: tokens held, pairs of tokens, tokens appended
        new, past = _lengths(c)
        held = sum(n + p for n, p in zip(new, past))
        pairs = c["batch"] * max(new) * (max(new) + max(past)) * c["q_heads"]
        if held * kv * dim <= 1 << 30 and pairs <= 4e9 and sum(new) <= 16411:
            return c
        if c["batch"] > 1:
            c["batch"] = (c["batch"] + 1) // 2
        elif c["past_hi"] > 4:
            c["past_lo"], c["past_hi"] = c["past_lo"] // 2, c["past_hi"] // 2
        else:
            c["new_lo"], c["new_hi"] = max(1, c["new_lo"] // 2), max(1, c["new_hi"] // 2)


def _lengths(c):
    r = random.Random(c["lens"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    return new, [r.randint(c["past_lo"], c["past_hi"]) for _ in range(c["batch"])]


def _visible(c, p):
    """How many tokens the token at position p sees."""
    if not c["window"]:
        return p + 1
    lo = max(0, p + 1 - c["window"])
    return p + 1 - lo + min(c["sinks"], lo)


def work(case):
    c = case
    new, past = _lengths(c)
    T, d, per = sum(new), c["dim"], c["kv_heads"] * c["dim"]
    held = per * 2 if c["bits"] == 16 else per // 2 + per // 16      # bytes of one token's keys (or values) in the cache
    q = T * c["q_heads"] * d * 2
    if c["op"] == "append":
        nbytes = 2 * q + T * (2 * per * 2 + 2 * held + 4 * c["rot"])
        flops = 3 * T * (c["q_heads"] + c["kv_heads"]) * c["rot"]
        if c["bits"] == 4:                                           # and read back as the values it stands for
            nbytes += T * (2 * held + 2 * per * 2)
        return {"bytes": nbytes, "flops": flops}
    pairs = read = 0
    for n, p in zip(new, past):
        pairs += sum(_visible(c, t) for t in range(p, p + n))
        if c["window"]:
            lo = max(0, p + 1 - c["window"])                          # the first new token's window reaches back furthest
            read += p + n - lo + min(c["sinks"], lo)
        else:
            read += p + n
    return {"bytes": 2 * q + T * c["q_heads"] * 4 + 2 * held * read, "flops": 4 * pairs * c["q_heads"] * d}


def prepare(case, seed):
    c = case
    new, past = _lengths(c)
    g = torch.Generator(device=DEV).manual_seed(seed)
    T, B, d, kv, page = sum(new), c["batch"], c["dim"], c["kv_heads"], c["page"]
    pages = [-(-(n + p) // page) for n, p in zip(new, past)]
    count = sum(pages) + 3
    order = torch.randperm(count, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(B, max(pages), dtype=torch.int32, device=DEV)
    at = torch.arange(max(pages), device=DEV)[None, :]
    held = torch.tensor(pages, device=DEV)
    first = torch.cumsum(held, 0) - held
    table[at < held[:, None]] = order[(first[:, None] + at)[at < held[:, None]]]
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(torch.tensor(new, device=DEV), 0)

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0, std, generator=g)

    s = dict(case=dict(c), q=normal(T, c["q_heads"], d, std=2.0), table=table, longest=max(n + p for n, p in zip(new, past)), most=max(new),
             cu=None if c["new_hi"] == 1 else cu, lens=torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32, device=DEV))
    shape = (count, kv, page, d)
    k, v = normal(*shape), normal(*shape)
    if c["bits"] == 16:
        s["cache"] = (k, v, None, None)
    else:
        (kc, ks), (vc, vs) = _to_four(k), _to_four(v)
        s["cache"] = (kc, vc, ks, vs)
    if c["op"] == "append":
        s["k"], s["v"] = normal(T, kv, d), normal(T, kv, d)
        # the rotations of each position: cosines, then sines, with 16 significant bits, so that a product with a
        # bfloat16 value is exact in 32 bits
        f = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
        a = torch.arange(s["longest"], dtype=torch.float64, device=DEV)[:, None] * f
        m, e = torch.frexp(torch.cat([torch.cos(a), torch.sin(a)], 1))
        s["rope"] = torch.ldexp(torch.round(m * 65536), e - 16).float().contiguous()
    return s


# ---- the plain form ---------------------------------------------------------------------------------

def _to_four(x):
    """Two values a byte, and a scale for each 16 of them."""
    v = x.float().unflatten(-1, (-1, 16))
    s = (v.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    f = s.float()[..., None]
    y = torch.where(f > 0, v.abs() / f, torch.zeros_like(v))
    code = ((y > 0.25).byte() + (y >= 0.75).byte() + (y > 1.25).byte() + (y >= 1.75).byte() + (y > 2.5).byte() + (y >= 3.5).byte() + (y > 5).byte())
    code = (code + 8 * torch.signbit(v).byte()).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s


def _of_four(code, s):
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=code.device)
    x = torch.stack([level[(code & 15).long()], level[(code >> 4).long()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * s.float()[..., None]).flatten(-2)


def _owners(s, T):
    """For each token its request, and its position there."""
    t = torch.arange(T, device=DEV)
    if s["cu"] is None:
        return t, s["lens"].long() - 1
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, s["lens"].long()[b] - cu[b + 1] + t


def _rotated(x, cs, c):
    r, x = c["rot"], x.float()
    cos, sin = cs[:, None, : r // 2], cs[:, None, r // 2:]
    y = x.clone()
    first, second = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y.bfloat16()


def _append(s):
    c = s["case"]
    b, at = _owners(s, s["k"].shape[0])
    cs = s["rope"][at]
    q, k, v = _rotated(s["q"], cs, c), _rotated(s["k"], cs, c), s["v"]
    page, row = s["table"][b, at // c["page"]].long(), at % c["page"]
    kc, vc, ks, vs = s["cache"]
    if c["bits"] == 16:
        kc[page, :, row], vc[page, :, row] = k, v
        return q, kc, vc
    (k4, k8), (v4, v8) = _to_four(k), _to_four(v)
    kc[page, :, row], vc[page, :, row] = k4, v4
    ks.view(torch.uint8)[page, :, row], vs.view(torch.uint8)[page, :, row] = k8.view(torch.uint8), v8.view(torch.uint8)
    return q, _of_four(k4, k8).bfloat16(), _of_four(v4, v8).bfloat16()


def _attend(s):
    c = s["case"]
    T, kv, d, most, B = s["q"].shape[0], c["kv_heads"], c["dim"], s["most"], c["batch"]
    kc, vc, ks, vs = s["cache"]
    J = s["table"].shape[1] * c["page"]

    def whole(x, scales):  # [B][kv heads][tokens][channels], in 32 bits
        x = x[s["table"].long()].transpose(1, 2).flatten(2, 3)
        return x.float() if scales is None else _of_four(x, scales.view(torch.uint8)[s["table"].long()].transpose(1, 2).flatten(2, 3).view(torch.float8_e4m3fn))

    k, v = whole(kc, ks), whole(vc, vs)
    lens = s["lens"].long()
    start = torch.arange(B, device=DEV) if s["cu"] is None else s["cu"][:-1].long()
    count = torch.ones(B, dtype=torch.long, device=DEV) if s["cu"] is None else s["cu"].long().diff()
    i = torch.arange(most, device=DEV)
    token = (start[:, None] + i).clamp(max=T - 1)
    q = s["q"][token].float().view(B, most, kv, -1, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    p = (lens - count)[:, None] + i                                      # [B][most]: positions
    j = torch.arange(J, device=DEV)
    see = (j <= p[..., None]) & (i < count[:, None])[..., None]
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    see = see[:, None, None]
    x = (q @ k.transpose(2, 3)).mul_(d ** -0.5).view(B, kv, -1, most, J).masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v).view(B, kv, -1, most, d) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2, 3)
    owner, at = _owners(s, T)
    return o[owner, at - (lens - count)[owner]].bfloat16(), lse[owner, at - (lens - count)[owner]].contiguous()


def run(state):
    s, c = state, state["case"]
    if not own:
        return _append(s) if c["op"] == "append" else _attend(s)
    import kda_gated_delta_gb300 as kda
    if c["op"] == "attend":
        return kda.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu"], window=c["window"], sinks=c["sinks"],
                                   max_new=s["most"], max_len=s["longest"], return_lse=True)
    q = kda.kv_append(s["k"], s["v"], s["cache"], s["table"], s["lens"], s["cu"], q=s["q"], rope=s["rope"], interleaved=c["interleaved"])
    if c["bits"] == 16:
        return (q,) + s["cache"][:2]
    return (q,) + kda.kv_read(s["cache"], s["table"], s["lens"], s["cu"], num_tokens=s["k"].shape[0])


# ---- the definition, in 64 bits ----------------------------------------------------------------------

def _four_exact(x):
    """The values that 4 bits hold for bfloat16 x, by the spacing of the grids instead of their borders."""
    x = x.double().unflatten(-1, (-1, 16))
    a = (x.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)        # e4m3: 3 mantissa bits, smallest exponent -6
    scale = torch.round(a / step) * step                                        # to nearest, ties to even
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(1.0, 6.0))) - 1)       # e2m1: 1 mantissa bit, smallest exponent 0
    return ((torch.round(y / step) * step).clamp(-6, 6) * scale).flatten(-2)


def _turned_exact(x, cos, sin, c):
    r = c["rot"]
    x = x.double()
    z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else torch.complex(x[..., : r // 2], x[..., r // 2: r])
    z = z * torch.complex(cos, sin)[:, None]
    y = torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., r:]], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    new, past = _lengths(c)
    kc, vc, ks, vs = s["cache"]
    if c["op"] == "append":
        at = torch.cat([torch.arange(p, p + n, device=DEV) for n, p in zip(new, past)])
        cs = s["rope"].double()[at]
        cos, sin = cs.chunk(2, 1)
        q, k = _turned_exact(s["q"], cos, sin, c), _turned_exact(s["k"], cos, sin, c)
        if c["bits"] == 4:  # what a key is held as goes by the key in bfloat16
            return q, _four_exact(k.bfloat16()), _four_exact(s["v"])
        if kc.numel() > 1 << 30:
            return None
        kc, vc, n0 = kc.double(), vc.double(), 0
        for i, (n, p) in enumerate(zip(new, past)):
            t = torch.arange(p, p + n, device=DEV)
            page = s["table"][i].long()[t // c["page"]]
            kc[page, :, t % c["page"]], vc[page, :, t % c["page"]] = k[n0:n0 + n], s["v"][n0:n0 + n].double()
            n0 += n
        return q, kc, vc
    group, n0, outs, lses = c["q_heads"] // c["kv_heads"], 0, [], []
    for i, (n, p) in enumerate(zip(new, past)):
        t = torch.arange(p + n, device=DEV)
        if c["window"]:
            t = t[(t < c["sinks"]) | (t > p - c["window"])]
        rows = (s["table"][i].long()[t // c["page"]], t % c["page"])
        o = torch.empty(n, c["q_heads"], c["dim"], dtype=torch.float64, device=DEV)
        lse = torch.empty(n, c["q_heads"], dtype=torch.float64, device=DEV)
        pos = torch.arange(p, p + n, device=DEV)[:, None]
        hidden = (t > pos) | (((t <= pos - c["window"]) & (t >= c["sinks"])) if c["window"] else False)
        for h in range(c["kv_heads"]):
            def rows_of(x, scales):
                if scales is None:
                    return x[rows[0], h, rows[1]].double()
                y = x[rows[0], h, rows[1]].long()
                level = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
                y = torch.stack([y % 16, y // 16], -1).flatten(1)
                y = level[y % 8] * (1 - 2 * (y // 8))
                return y * scales.view(torch.uint8)[rows[0], h, rows[1]].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
            k, v = rows_of(kc, ks), rows_of(vc, vs)
            for r in range(h * group, h * group + group):
                x = (s["q"][n0:n0 + n, r].double() @ k.T) / math.sqrt(c["dim"])
                x[hidden] = -math.inf
                lse[:, r] = torch.logsumexp(x, 1)
                o[:, r] = torch.exp(x - lse[:, r, None]) @ v
        outs.append(o)
        lses.append(lse)
        n0 += n
    return torch.cat(outs), torch.cat(lses)
