"""Plain 64-bit forms of the operators around a recurrence (short convolution, selective recurrence, group norm),
with the sums of magnitudes that their error bounds are stated in.  Everything on the CPU."""
import torch


def half_step(dtype):
    """A rounding to `dtype` is off by at most this share of the value."""
    return torch.finfo(dtype).eps / 2


F32 = half_step(torch.float32)


def lengths_to_cu(lens, device="cpu"):
    return torch.tensor([0] + list(lens)).cumsum(0).to(device=device, dtype=torch.int32)


def conv(x, weight, pool, slots, lens, bias=None, silu=False):
    """(outputs, new pool, sum of magnitudes) for requests of `lens` tokens, slot < 0: padding."""
    x, w, pool = x.double().cpu(), weight.double().cpu(), pool.double().cpu().clone()
    y, mag, at = torch.zeros_like(x), torch.zeros_like(x), 0
    for slot, n in zip(slots, lens):
        if slot >= 0 and n > 0:
            line = torch.cat([pool[slot], x[at:at + n]])
            for t in range(n):
                taps = line[t:t + w.shape[1]].T * w
                y[at + t] = taps.sum(1) + (0 if bias is None else bias.double().cpu())
                mag[at + t] = taps.abs().sum(1) + (0 if bias is None else bias.double().cpu().abs())
            pool[slot] = line[-(w.shape[1] - 1):]
        at += n
    return (y * torch.sigmoid(y) if silu else y), pool, mag


def ssm(x, dt, B, C, A_log, pool, slots, lens, dt_bias=None, D=None):
    """(outputs, new pool, the same two with every product's magnitude in its place)."""
    x, dt, B, C, A = x.double().cpu(), dt.double().cpu(), B.double().cpu(), C.double().cpu(), A_log.double().cpu().exp()
    H, G = x.shape[1], B.shape[1]
    D = torch.zeros(H, dtype=torch.float64) if D is None else D.double().cpu()
    dt = dt + (0 if dt_bias is None else dt_bias.double().cpu())
    dt = torch.where(dt > 20, dt, torch.log1p(torch.exp(dt)))
    B, C = B.repeat_interleave(H // G, 1), C.repeat_interleave(H // G, 1)
    pool = pool.double().cpu().clone()
    mags = pool.abs()
    y, y_mag, at = torch.zeros_like(x), torch.zeros_like(x), 0
    for slot, n in zip(slots, lens):
        if slot >= 0:
            for t in range(at, at + n):
                a = torch.exp(-dt[t] * A)[:, None, None]
                u = (dt[t][:, None] * x[t])[:, :, None]
                pool[slot] = a * pool[slot] + u * B[t][:, None, :]
                mags[slot] = a * mags[slot] + u.abs() * B[t].abs()[:, None, :]
                y[t] = (pool[slot] * C[t][:, None, :]).sum(-1) + D[:, None] * x[t]
                y_mag[t] = (mags[slot] * C[t].abs()[:, None, :]).sum(-1) + (D[:, None] * x[t]).abs()
        at += n
    return y, pool, y_mag, mags


def act(x, name):
    return x if name is None else torch.sigmoid(x) * (x if name == "silu" else 1)


def norm(x, weight=None, bias=None, gate=None, activation=None, gate_first=False, center=True, eps=1e-5):
    x = x.double().cpu()
    gate = None if gate is None else act(gate.double().cpu(), activation)
    if gate_first:
        x = x * gate
    if center:
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double().cpu()
    if bias is not None:
        y = y + bias.double().cpu()
    return act(y, activation) if gate is None else y if gate_first else y * gate


def within(got, want, bound):
    """Every element within its bound; the message gives the worst."""
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape, (got.shape, want.shape)
    bound = torch.as_tensor(bound, dtype=torch.float64).expand_as(want)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        i = int(torch.where(bad, off / bound.clamp(min=1e-300), torch.zeros(())).nan_to_num(nan=float("inf")).argmax())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} elements off; the worst, number {i}: got {got.flatten()[i]:.9g}, "
                             f"want {want.flatten()[i]:.9g}, bound {bound.flatten()[i]:.3g}")
