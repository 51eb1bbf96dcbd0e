"""Plain 64-bit implementations for pools held in 4 bits: codes, scales and tiles.  Host only."""
import numpy as np
import torch

from tests import block8_ref as R

BS = 16
CODES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
TOP = 61440.0


def scales_of(byte):
    """Values of scale bytes: 5 exponent bits of bias 15, 3 mantissa bits."""
    b = np.asarray(byte, np.int64)
    e, m = b >> 3, b & 7
    return np.where(e > 0, (8 + m) * 2.0 ** (e - 18), m * 2.0 ** -17)


SCALES = scales_of(np.arange(0xE3))              # up to 10240


def _nearest(x, values):
    """Index of the nearest value; of two the even one."""
    up = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    below, above = x - values[up - 1], values[up] - x
    return np.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)


def encode(x):
    """Rows [..., D] in 64 bits -> signed code values [..., D] and scale bytes [..., D / 16].  Units
    with a NaN have the byte 0xff and zeros."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 16)
    bad = np.isnan(g).any(-1)
    g = np.where(bad[..., None], 0.0, g)
    amax = np.abs(g).max(-1)
    byte = _nearest(np.minimum(amax, 4 * TOP) / 6, SCALES)
    byte = np.where(amax > 0, np.maximum(byte, 1), 0)
    s = np.where(byte > 0, SCALES[byte], 1.0)[..., None]
    code = np.sign(g) * CODES[_nearest(np.minimum(np.abs(g), 4 * TOP) / s, CODES)]
    return code.reshape(x.shape), np.where(bad, 0xFF, byte).astype(np.uint8)


def values_of(code, byte):
    s = np.where(byte == 0xFF, np.nan, scales_of(byte))
    return (code.reshape(*byte.shape, 16) * s[..., None]).reshape(code.shape)


def pack(code, byte):
    """Codes [..., 16, D] and scale bytes [..., 16, D / 16] -> tiles, uint8 [..., 16, 9 D / 16]."""
    n = np.searchsorted(CODES, np.abs(code)) + 8 * (code < 0)
    b = (n[..., 0::2] | (n[..., 1::2] << 4)).astype(np.uint8)
    D, lead = code.shape[-1], code.shape[:-2]
    tile = np.concatenate([b.reshape(*lead, -1), byte.reshape(*lead, -1)], -1)
    return torch.from_numpy(tile.reshape(*lead, BS, 9 * D // 16))


def unpack(pool):
    """Tiles -> (codes, scale bytes, values), [..., 16, D]."""
    t = pool.cpu().numpy()
    D, lead = t.shape[-1] * 16 // 9, t.shape[:-2]
    t = t.reshape(*lead, 9 * D)
    b = t[..., :8 * D].reshape(*lead, BS, D // 2)
    n = np.stack([b & 15, b >> 4], -1).reshape(*lead, BS, D).astype(np.int64)
    code = CODES[n & 7] * (1 - 2 * (n >> 3))
    byte = t[..., 8 * D:].reshape(*lead, BS, D // 16)
    return code, byte, values_of(code, byte)


def pool(g, blocks, heads, dim, spread=1.0):
    """A random pool (uint8 tensor)."""
    x = torch.randn(blocks, heads, BS, dim, generator=g, dtype=torch.float64)
    x *= torch.exp2(spread * torch.randn(blocks, heads, BS, 1, generator=g, dtype=torch.float64))
    return pack(*encode(x.numpy()))


class Batch:
    """Pools, tables and lengths; rows that hold no token have NaN scales."""

    def __init__(self, seed, lens, hkv, dim, spread=1.0, width=None, spare=3, poison=True):
        g = self.g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.dim = np.asarray(lens, np.int32), hkv, dim
        self.tables, self.blocks = R.tables_for(g, lens, spare=spare, width=width)
        self.kc, self.vc = pool(g, self.blocks, hkv, dim, spread), pool(g, self.blocks, hkv, dim, spread)
        self.live = np.zeros((self.blocks, BS), bool)
        for b, n in enumerate(lens):
            for p in range(int(n)):
                self.live[self.tables[b, p // BS], p % BS] = True
        if poison:
            for t in (self.kc, self.vc):
                self.scales(t)[torch.from_numpy(~self.live)[:, None].expand(-1, hkv, -1)] = 0xFF

    def scales(self, t):
        """The scale bytes of a pool as a view [blocks][heads][16][dim / 16]."""
        return t.view(self.blocks, self.hkv, -1)[:, :, 8 * self.dim:].unflatten(-1, (BS, self.dim // 16))

    def device(self):
        return [self.kc.cuda(), self.vc.cuda(), torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.lens).cuda()]

    def query(self, rows, hq):
        return torch.randn(rows, hq, self.dim, generator=self.g).to(torch.bfloat16)

    def reference(self, q, rows, scale=None, window=0, floor=1.0):
        """q [rows][Hq][D] float64; rows: (sequence, last position) of each.  Output and the error a
        kernel may make beside the output's own rounding (block8_ref.attention, scales of one)."""
        group, scale = q.shape[1] // self.hkv, self.dim ** -0.5 if scale is None else scale
        kv, vv = unpack(self.kc)[2], unpack(self.vc)[2]
        one = np.ones(self.blocks)
        out, bound = np.zeros_like(q), np.zeros_like(q)
        for i, (b, last) in enumerate(rows):
            lo = max(0, last + 1 - window) if window else 0
            for h in range(self.hkv):
                j = slice(h * group, (h + 1) * group)
                out[i, j], bound[i, j] = R.attention(q[i, j], kv[:, h], one, vv[:, h], one, self.tables[b], lo, last + 1,
                                                     scale, floor)
        return out, bound


def check(got, ref, bound, what=""):
    err = np.abs(got.double().cpu().numpy() - ref)
    limit = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    assert (err <= limit).all(), (what, float(np.nanmax(err - limit)), np.argwhere(~(err <= limit))[:4].tolist())
