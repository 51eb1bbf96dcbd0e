"""Plain 64-bit implementations of the step operators (plan, rotary positions with the cache
write, attention over E4M3 pools with block scales), and inputs for them.  Host only."""
import math

import numpy as np
import torch

BS = 16


def plan(tables, lens, new, free, num_free, capacity, num_blocks):
    """pa_plan_step, sequence by sequence.  Returns new arrays."""
    tables = tables.copy()
    B, width = tables.shape
    out, start, slots, pos = lens.copy(), [0], [], []
    left, stopped = num_free, False
    for b in range(B):
        L, T = int(lens[b]), int(new[b])
        ok = not (L < 0 or T < 0 or L + T > width * BS)
        T = T if ok else 0
        need = -(-(L + T) // BS) - -(-L // BS) if T else 0
        if stopped or need > left or len(slots) + T > capacity:
            stopped = stopped or T > 0
            start.append(len(slots))
            continue
        for j in range(need):
            left -= 1
            tables[b, -(-L // BS) + j] = free[left]
        for p in range(L, L + T):
            phys = int(tables[b, p // BS])
            slots.append(phys * BS + p % BS if 0 <= phys < num_blocks else -1)
            pos.append(p)
        out[b] = L + T
        start.append(len(slots))
    fill = capacity - len(slots)
    return (tables, out, np.array(start, np.int32), np.array(slots + [-1] * fill, np.int64),
            np.array(pos + [0] * fill, np.int32), left)


def rotary_angles(pos, rot, base=10000.0, scaling="none", factor=1.0, original=4096, fast=32.0, slow=1.0):
    """cos, sin [tokens][rot / 2] in float64, the attention factor included."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    theta = base ** (-2.0 * i / rot) if rot else i
    a = 1.0
    if scaling == "linear":
        theta = theta / factor
    if scaling == "by_parts":
        idx = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(idx(fast)), 0), min(math.ceil(idx(slow)), rot - 1)
        r = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        theta = theta * (1 - r) + theta / factor * r
        a = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    ang = np.asarray(pos, np.float64)[:, None] * theta
    return a * np.cos(ang), a * np.sin(ang)


def rotate(x, cos, sin, interleaved):
    """x [tokens][heads][D] float64 turned; and per element |x0| + |x1| of its pair (0 behind)."""
    half = cos.shape[1]
    y, mass = x.copy(), np.zeros_like(x)
    if half:
        i0 = np.arange(half) * 2 if interleaved else np.arange(half)
        i1 = i0 + 1 if interleaved else i0 + half
        a, b, c, s = x[..., i0], x[..., i1], cos[:, None], sin[:, None]
        y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
        mass[..., i0] = mass[..., i1] = np.abs(a) + np.abs(b)
    return y, mass


def block_scale(amax):
    """Smallest 2^e, e in [-32, 31], with amax <= 448 * 2^e."""
    for e in range(-32, 32):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 31


def e4m3(x):
    """float64 -> nearest E4M3 value, ties to even, saturating (values, float64)."""
    a = np.abs(x)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    step = 2.0 ** (np.clip(e, -6, 8) - 3)
    return np.sign(x) * np.minimum(np.round(a / step) * step, 448.0)   # np.round: half to even


def decode_codes(t):
    """E4M3 codes (uint8 or float8 tensor) as float64 values."""
    return t.cpu().view(torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def encode(x):
    """float64 array of E4M3 values -> uint8 codes."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)


def write_blocks(rows, slots, values, scales):
    """Block-scaled write of rows [tokens][heads][D] into value arrays [blocks][heads][16][D] and
    scales [blocks][heads], in place."""
    by_block = {}
    for i, s in enumerate(slots):
        if 0 <= s < values.shape[0] * BS:
            by_block.setdefault(int(s) // BS, {})[int(s) % BS] = i
    for blk, offs in by_block.items():
        low = min(offs)
        for h in range(values.shape[1]):
            x = {o: rows[i, h] for o, i in offs.items()}
            scale = block_scale(max(float(np.nanmax(np.abs(v), initial=0.0)) for v in x.values()))
            if low:
                scale = max(scale, float(scales[blk, h]))
                values[blk, h, :low] = e4m3(values[blk, h, :low] * (scales[blk, h] / scale))
            for o, v in x.items():
                values[blk, h, o] = e4m3(v / scale)
            scales[blk, h] = scale


def attention(q, kv, ks, vv, vs, table, lo, hi, scale, floor=1.0):
    """One query group [g][D] over positions [lo, hi) of one sequence and KV head: output, and the
    error a kernel may make beside the output's own rounding.  kv, vv: code values
    [blocks][16][D] of the head, ks, vs its scales [blocks].

    The weights w = 2^(s + log2 sv - m) are rounded to f16: 2^-11 of each, or 2^-25 where w is below
    f16's normal range, in units in which the largest is at least 1 (floor: the decode kernel's case;
    prefill's largest is at least 1/2 and a weight may be rounded again when a later reference scales
    it: floor 4).  f32 sums and 2^x add less than 2^-15 of the weighted magnitudes."""
    if hi <= lo:
        return np.zeros_like(q), np.zeros_like(q)
    pos = np.arange(lo, hi)
    blk, off = np.asarray(table)[pos // BS], pos % BS
    k, v = kv[blk, off] * ks[blk][:, None], vv[blk, off] * vs[blk][:, None]
    s = q @ k.T * scale
    p = np.exp(s - s.max(-1, keepdims=True))
    l = p.sum(-1, keepdims=True)
    out, mass = p @ v / l, p @ np.abs(v) / l
    w = p * vs[blk]
    tail = floor * 2.0 ** -25 * w.max(-1, keepdims=True) / l * np.abs(vv[blk, off]).sum(0)
    return out, (2.0 ** -11 + 2.0 ** -15) * mass + tail


def pools(g, blocks, heads, dim, spread=1.5):
    """Random E4M3 pool: codes (uint8 tensor) and power-of-two scales (float32 tensor)."""
    x = torch.randn(blocks, heads, BS, dim, generator=g, dtype=torch.float64)
    x *= torch.exp2(spread * torch.randn(blocks, heads, 1, 1, generator=g, dtype=torch.float64))
    s = torch.tensor([[block_scale(float(x[b, h].abs().max())) for h in range(heads)] for b in range(blocks)],
                     dtype=torch.float64)
    return (x / s[:, :, None, None]).float().to(torch.float8_e4m3fn).view(torch.uint8), s.float()


def tables_for(g, lens, spare=3, width=None):
    need = [-(-int(n) // BS) for n in lens]
    blocks = sum(need) + spare
    perm = torch.randperm(blocks, generator=g).numpy()
    width = width or max(1, max(need))
    t, at = np.full((len(need), width), -1, np.int32), 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, blocks
