"""Pools held in 4 bits: pa_rope_cache_write_fp4, pa_cache_read_fp4, pa_decode_fp4 and
pa_prefill_fp4 against 64-bit implementations; codes, scales and values read back bit for bit."""
import numpy as np
import pytest
import torch

from tests import block8_ref as R
from tests import fp4_ref as F

pytestmark = pytest.mark.gpu

# cos and sin: the angle is held to 2^-24 of at most half a turn (pi 2^-24 < 2^-22 radians), sincospi
# to 2 units of 2^-23; two products and a sum of f32 round 3 times 2^-24.  Per |x0| + |x1|:
TURN = 2.0 ** -22 + 2.0 ** -22 + 3 * 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_100_gb300.build import build
    build()
    import paged_kv_cache_100_gb300 as m
    return m


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _angles(rope, pos):
    """cos and sin (64 bits) of the plan's own fractions of a turn, exact at any position."""
    turns = [int(t) % (1 << 64) for t in rope.turns.cpu().tolist()]
    frac = np.array([[((int(p) * t) % (1 << 64)) / 2.0 ** 64 for t in turns] for p in pos]).reshape(len(pos), len(turns))
    return rope.attention_factor * np.cos(2 * np.pi * frac), rope.attention_factor * np.sin(2 * np.pi * frac)


def _written(pool, rows, slots):
    """The pool after the write of rows [tokens][heads][D] (64 bits): codes and scale bytes."""
    code, byte, _ = F.unpack(pool)
    c, b = F.encode(rows)
    for i, s in enumerate(slots):
        if 0 <= s < pool.shape[0] * 16:
            code[s // 16, :, s % 16], byte[s // 16, :, s % 16] = c[i], b[i]
    return code, byte


def _same(pool, want, what):
    code, byte, _ = F.unpack(pool)
    assert np.array_equal(byte, want[1]), (what, "scales", np.argwhere(byte != want[1])[:4].tolist())
    assert np.array_equal(code, want[0]), (what, "codes", np.argwhere(code != want[0])[:4].tolist())


# ---------------------------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (128, 64), (128, 20), (64, 2), (256, 250), (96, 96), (80, 0), (16, 16),
                                   (48, 46), (256, 256)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 2), (37, 3, 3)])
def test_write_matches(pkv, D, rot, dtype, interleaved, T, Hq, Hkv):
    g = torch.Generator().manual_seed(D + rot + T)
    blocks = 5
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g) * torch.exp2(2 * torch.randn(T, Hq + 2 * Hkv, 1, generator=g))
    qkv = qkv.to(dtype)
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32)
    slots = torch.randperm(blocks * 16, generator=g)[:T]
    if T > 3:
        slots[3] = -1
    kc, vc = F.pool(g, blocks, Hkv, D), F.pool(g, blocks, Hkv, D)
    rope = pkv.rotary_plan(rot, interleaved=interleaved)
    x, kd, vd, status = qkv.cuda(), kc.cuda(), vc.cuda(), _status()
    args = (x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos.cuda(), rope, kd, vd, slots.cuda())
    out = pkv.rope_cache_write_fp4(x[:, :Hq], *args, status=status)
    cos, sin = _angles(rope, pos.tolist())
    ref, mass = R.rotate(qkv.double().numpy(), cos, sin, interleaved)
    err = np.abs(out.double().cpu().numpy() - ref[:, :Hq])
    m = mass[:, :Hq]
    assert (err <= TURN * m + HALF_STEP[dtype] * (np.abs(ref[:, :Hq]) + TURN * m)).all()
    _same(kd, _written(kc, ref[:, Hq:Hq + Hkv], slots.tolist()), "keys")
    _same(vd, _written(vc, qkv[:, Hq + Hkv:].double().numpy(), slots.tolist()), "values")
    assert int(status.item()) == 0
    # in place on contiguous queries, and without queries
    q = x[:, :Hq].contiguous()
    again = pkv.rope_cache_write_fp4(q, *args, query_out=q)
    assert again is q and torch.equal(q, out)
    k2, v2 = kc.cuda(), vc.cuda()
    assert pkv.rope_cache_write_fp4(None, *args[:4], k2, v2, args[6]) is None
    assert torch.equal(k2, kd) and torch.equal(v2, vd)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_of_borders_and_extremes(pkv, dtype):
    """Elements on and beside the borders of two codes and of two scales, and magnitudes of every size."""
    D, rows = 64, []
    rng = np.random.default_rng(5)
    tie = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for byte in list(range(1, 30)) + list(range(100, 140)) + [0xE0, 0xE1, 0xE2]:
        s = F.SCALES[byte]
        rows.append(np.concatenate([[6 * s], rng.choice(tie, 15) * s * rng.choice([-1, 1], 15)]))
    mid = (F.SCALES[1:] + F.SCALES[:-1]) / 2 * 6                     # amax between two scales: ties to even
    for m in mid:
        rows.append(np.concatenate([[m], rng.uniform(-1, 1, 15) * m]))
    for e in range(-40, 17):
        rows.append(rng.standard_normal(16) * 2.0 ** e)
    rows += [np.zeros(16), np.full(16, -0.0), np.full(16, 2.0 ** -133), np.full(16, 61440.0)]
    x = np.stack(rows)
    x = np.concatenate([x, np.zeros((-len(x) % 4, 16))]).reshape(-1, 1, D)
    t = torch.from_numpy(x).to(dtype)
    if dtype == torch.float32:                                       # and one step of f32 beside the borders
        t = torch.cat([t, torch.nextafter(t, t * 2), torch.nextafter(t, t * 0)])
    T = t.shape[0]
    blocks = -(-T // 16)
    kc, vc, status = pkv.fp4_pool(blocks, 1, D), pkv.fp4_pool(blocks, 1, D), _status()
    slots = torch.arange(T).cuda()
    pkv.rope_cache_write_fp4(None, t.cuda(), t.cuda(), None, None, kc, vc, slots, status=status)
    want = _written(torch.zeros_like(vc).cpu(), t.double().numpy(), range(T))
    _same(vc, want, "values")
    _same(kc, want, "keys")                                          # not turned
    assert int(status.item()) == (256 if (t.abs() > 61440).any() else 0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_of_many_turned_keys(pkv, dtype, interleaved):
    """Half a million turned keys, some pairs of very unlike halves: codes and scales of the exact rotation."""
    g = torch.Generator().manual_seed(11)
    T, H, D = 1000, 4, 128
    k = torch.randn(T, H, D, generator=g)
    k[:, 1, :64] *= 2.0 ** 14                                        # partners far larger than their own unit
    k[:, 2] *= torch.exp2(4 * torch.randn(T, D, generator=g))
    k = k.to(dtype)
    pos = torch.randint(0, 1 << 30, (T,), generator=g, dtype=torch.int32)
    rope = pkv.rotary_plan(D, 500000.0, interleaved=interleaved, scaling="by_parts", factor=8.0)
    blocks = -(-T // 16)
    kc, vc = pkv.fp4_pool(blocks, H, D), pkv.fp4_pool(blocks, H, D)
    slots = torch.randperm(blocks * 16, generator=g)[:T]
    pkv.rope_cache_write_fp4(None, k.cuda(), k.cuda(), pos.cuda(), rope, kc, vc, slots.cuda())
    cos, sin = _angles(rope, pos.tolist())
    ref, _ = R.rotate(k.double().numpy(), cos, sin, interleaved)
    zero = torch.zeros(kc.shape, dtype=torch.uint8)
    _same(vc, _written(zero, k.double().numpy(), slots.tolist()), "values")
    _same(kc, _written(zero, ref, slots.tolist()), "keys")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 64, False), (128, 64, True), (128, 94, True), (128, 94, False), (256, 96, False),
                                               (160, 32, False), (64, 64, False), (224, 224, True)])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("by_parts", 32.0)])
def test_write_of_partly_turned_keys_and_at_position_zero(pkv, D, rot, interleaved, dtype, scaling, factor):
    """Units that are turned beside units that are not; tokens at position 0, where bf16 elements are borders of codes."""
    g = torch.Generator().manual_seed(D + rot)
    T, H = 300, 3
    k = (torch.randn(T, H, D, generator=g) * torch.exp2(3 * torch.randn(T, H, 1, generator=g))).to(dtype)
    pos = torch.randint(0, 3000, (T,), generator=g, dtype=torch.int32)
    pos[::5] = 0
    rope = pkv.rotary_plan(rot, interleaved=interleaved, scaling=scaling, factor=factor)
    blocks = 20
    kc, vc = pkv.fp4_pool(blocks, H, D), pkv.fp4_pool(blocks, H, D)
    slots = torch.randperm(blocks * 16, generator=g)[:T]
    pkv.rope_cache_write_fp4(None, k.cuda(), k.cuda(), pos.cuda(), rope, kc, vc, slots.cuda())
    ref, _ = R.rotate(k.double().numpy(), *_angles(rope, pos.tolist()), interleaved)
    zero = torch.zeros(kc.shape, dtype=torch.uint8)
    _same(vc, _written(zero, k.double().numpy(), slots.tolist()), "values")
    _same(kc, _written(zero, ref, slots.tolist()), "keys")


def test_write_of_unturned_f32_keys_beside_other_values(pkv):
    """Elements on and beside the borders of codes, in keys that are not the values: each row's codes are its own."""
    g = torch.Generator().manual_seed(21)
    T, H, D = 200, 3, 64
    tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    scale = torch.from_numpy(F.SCALES[8:0xE2])[torch.randint(0, 0xE2 - 8, (T, H, D // 16, 1), generator=g)].float()
    k = tie[torch.randint(0, 7, (T, H, D // 16, 16), generator=g)] * scale
    k *= torch.randint(0, 2, k.shape, generator=g) * 2 - 1
    beside = torch.randint(0, 3, k.shape, generator=g)
    k = torch.where(beside == 0, torch.nextafter(k, k * 2), torch.where(beside == 1, torch.nextafter(k, k * 0), k))
    k[..., 0] = 6 * scale[..., 0]
    k = k.reshape(T, H, D)
    v = torch.randn(T, H, D, generator=g)
    blocks = -(-T // 16)
    kc, vc = pkv.fp4_pool(blocks, H, D), pkv.fp4_pool(blocks, H, D)
    pkv.rope_cache_write_fp4(None, k.cuda(), v.cuda(), None, None, kc, vc, torch.arange(T).cuda())
    zero = torch.zeros(kc.shape, dtype=torch.uint8)
    _same(vc, _written(zero, v.double().numpy(), range(T)), "values")
    _same(kc, _written(zero, k.double().numpy(), range(T)), "keys")


def test_write_of_nan_and_infinity(pkv):
    D = 128
    x = torch.randn(4, 2, D, generator=torch.Generator().manual_seed(3))
    x[1, 0, 5], x[2, 1, 100], x[2, 1, 70] = float("nan"), float("inf"), -float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        t = x.to(dtype)
        kc, vc, status = pkv.fp4_pool(1, 2, D), pkv.fp4_pool(1, 2, D), _status()
        pkv.rope_cache_write_fp4(None, t.cuda(), t.cuda(), None, None, kc, vc, torch.arange(4).cuda(), status=status)
        _same(vc, _written(torch.zeros(vc.shape, dtype=torch.uint8), t.double().numpy(), range(4)), "values")
        assert torch.equal(kc, vc) and int(status.item()) == 256
        v = F.unpack(vc)[2][0]                                       # [heads][16][D]
        assert np.isnan(v[0, 1, :16]).all() and not np.isnan(v[0, 1, 16:]).any()
        assert v[1, 2, 100] == 61440 and v[1, 2, 70] == -61440
    # turned: what a NaN reaches is NaN, the rest of the row is not
    rope = pkv.rotary_plan(D)
    kc, vc = pkv.fp4_pool(1, 2, D), pkv.fp4_pool(1, 2, D)
    pkv.rope_cache_write_fp4(None, x.cuda(), x.cuda(), torch.ones(4, dtype=torch.int32).cuda(), rope, kc, vc, torch.arange(4).cuda())
    v = F.unpack(kc)[2][0]
    assert np.isnan(v[0, 1, :16]).all() and np.isnan(v[0, 1, 64:80]).all()
    assert not np.isnan(v[0, 1, 16:64]).any() and not np.isnan(v[0, 0]).any() and not np.isnan(v[0, 3]).any()


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("by_parts", 32.0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 20), (48, 48), (256, 96)])
def test_write_of_turned_keys_beyond_f32(pkv, D, rot, dtype, interleaved, scaling, factor):
    """Infinities that are turned, and finite pairs whose rotation leaves f32's range: saturated, with the sign of the exact
    rotation, in their own unit and in their partner's; a NaN only where the rotation is one."""
    g = torch.Generator().manual_seed(D + rot)
    T, H, half = 64, 2, rot // 2
    k = torch.randn(T, H, D, generator=g).to(dtype)
    top = torch.finfo(dtype).max
    inf = float("inf")
    odd = [(inf, 1.0), (-2.0, -inf), (top, top), (top, -top), (0.9 * top, 0.01 * top), (-top, 0.0), (0.0, top), (inf, inf),
           (inf, float("nan")), (0.75 * top, 0.7 * top), (1e30, -1e30)]
    for t in range(1, T):                                            # (the first token is ordinary)
        p = int(torch.randint(0, half, (1,), generator=g))
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        k[t, t % H, i], k[t, t % H, j] = odd[t % len(odd)]
    k[5, 1, rot - 2:] = 0
    pos = torch.randint(0, 3000, (T,), generator=g, dtype=torch.int32)
    pos[40:52] = 0                                                   # where nothing turns
    rope = pkv.rotary_plan(rot, interleaved=interleaved, scaling=scaling, factor=factor)
    kc, vc, status = pkv.fp4_pool(4, H, D), pkv.fp4_pool(4, H, D), _status()
    pkv.rope_cache_write_fp4(None, k.cuda(), k.cuda(), pos.cuda(), rope, kc, vc, torch.arange(T).cuda(), status=status)
    with np.errstate(invalid="ignore"):
        ref, _ = R.rotate(k.double().numpy(), *_angles(rope, pos.tolist()), interleaved)
    zero = torch.zeros(kc.shape, dtype=torch.uint8)
    _same(vc, _written(zero, k.double().numpy(), range(T)), "values")
    _same(kc, _written(zero, ref, range(T)), "keys")
    assert int(status.item()) == 256


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 64), (256, 96), (128, 36), (80, 80)])
def test_write_of_units_that_nearly_cancel(pkv, D, rot, dtype):
    """Units of which every element is turned into next to nothing: scales and codes of what is left, exactly."""
    g = torch.Generator().manual_seed(D + rot)
    T, H, half = 600, 2, rot // 2
    pos = torch.randint(1, 3000, (T,), generator=g, dtype=torch.int32)
    rope = pkv.rotary_plan(rot)
    cos, sin = (torch.from_numpy(x)[:, None] for x in _angles(rope, pos.tolist()))
    k = torch.randn(T, H, D, generator=g).to(dtype)
    # the pair's second element at random, of one size in a row; its first one nearest to what cancels
    second = (torch.randn(T, H, half, generator=g) * torch.exp2(20 * torch.rand(T, H, 1, generator=g))).to(dtype)
    k[..., half:rot] = second
    k[..., :half] = (second.double() * sin / torch.where(cos.abs() < 0.01, 1.0, cos)).to(dtype)
    blocks = -(-T // 16)
    kc, vc = pkv.fp4_pool(blocks, H, D), pkv.fp4_pool(blocks, H, D)
    pkv.rope_cache_write_fp4(None, k.cuda(), k.cuda(), pos.cuda(), rope, kc, vc, torch.arange(T).cuda())
    ref, mass = R.rotate(k.double().numpy(), cos[:, 0].numpy(), sin[:, 0].numpy(), False)
    if dtype == torch.float32:                                       # what is meant to be tested is there
        unit = slice(0, 16)
        assert (np.abs(ref[..., unit]).max(-1) < 2.0 ** -20 * mass[..., unit].max(-1)).mean() > 0.5
    zero = torch.zeros(kc.shape, dtype=torch.uint8)
    _same(kc, _written(zero, ref, range(T)), "keys")


@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (64, 64, True), (64, 20, False)])
def test_write_flags_the_exact_range(pkv, dim, rot, interleaved):
    """Elements turned into 61440 and a little more or less: flagged where the exact one is beyond it."""
    g = np.random.default_rng(rot)
    rope, T, half = pkv.rotary_plan(rot, interleaved=interleaved), 48, rot // 2
    pos = g.integers(1, 3000, T)
    cos, sin = _angles(rope, pos.tolist())
    k = np.zeros((T, 1, dim))
    for t in range(T):
        p = int(np.argmax(np.abs(cos[t])))                           # a pair that turns by little
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        k[t, 0, j] = np.float32(g.uniform(-500, 500))
        k[t, 0, i] = np.float32((61440.0 + k[t, 0, j] * sin[t, p]) / cos[t, p])
    ref, _ = R.rotate(k, cos, sin, interleaved)
    beyond = np.abs(ref).reshape(T, -1).max(-1) > 61440.0
    assert 10 < beyond.sum() < T - 10
    x, where = torch.from_numpy(k).float().cuda(), torch.from_numpy(pos).to(torch.int32).cuda()
    kc, vc, status = pkv.fp4_pool(T, 1, dim), pkv.fp4_pool(T, 1, dim), torch.zeros(T, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, 1, dim, device="cuda")
    for t in range(T):
        pkv.rope_cache_write_fp4(None, x[t:t + 1], zero, where[t:t + 1], rope, kc, vc, torch.tensor([t]).cuda(), status=status[t:t + 1])
    assert np.array_equal(status.cpu().numpy() == 256, beyond) and not (status.cpu().numpy() & ~256).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (64, 64, True), (64, 20, False)])
def test_write_of_turned_subnormal_keys(pkv, D, rot, interleaved, dtype):
    """Keys down to f32's last bit: a unit that is turned into anything but zero has a scale, as one of zeros has none."""
    g = torch.Generator().manual_seed(rot)
    T = 200
    size = torch.exp2(torch.randint(-150, -100, (T, 1, 1), generator=g).double())
    k = (torch.randn(T, 1, D, generator=g, dtype=torch.float64) * size * (torch.rand(T, 1, D, generator=g) < 0.1)).to(dtype)
    pos = torch.randint(0, 3000, (T,), generator=g, dtype=torch.int32)
    rope = pkv.rotary_plan(rot, interleaved=interleaved)
    blocks = -(-T // 16)
    kc, vc, status = pkv.fp4_pool(blocks, 1, D), pkv.fp4_pool(blocks, 1, D), _status()
    pkv.rope_cache_write_fp4(None, k.cuda(), k.cuda(), pos.cuda(), rope, kc, vc, torch.arange(T).cuda(), status=status)
    ref, _ = R.rotate(k.double().numpy(), *_angles(rope, pos.tolist()), interleaved)
    zero = torch.zeros(kc.shape, dtype=torch.uint8)
    _same(vc, _written(zero, k.double().numpy(), range(T)), "values")
    _same(kc, _written(zero, ref, range(T)), "keys")
    assert int(status.item()) == 0


def test_write_slots(pkv):
    """Slots past the pool are skipped and flagged, negative ones skipped; the query is turned all the same."""
    g = torch.Generator().manual_seed(8)
    x = torch.randn(5, 3, 64, generator=g).cuda()
    kc, vc = F.pool(g, 2, 1, 64), F.pool(g, 2, 1, 64)
    kd, vd, status = kc.cuda(), vc.cuda(), _status()
    rope = pkv.rotary_plan(64)
    pos = torch.arange(5, dtype=torch.int32).cuda()
    out = pkv.rope_cache_write_fp4(x[:, :1], x[:, 1:2], x[:, 2:], pos, rope, kd, vd,
                                   torch.tensor([-1, 32, 1 << 40, -(1 << 50), 1 << 62]).cuda(), status=status)
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc) and int(status.item()) == 4
    ref, _ = R.rotate(x[:, :1].double().cpu().numpy(), *_angles(rope, range(5)), False)
    assert np.allclose(out.double().cpu().numpy(), ref, atol=1e-5)
    # no token at all
    e = x[:0]
    assert pkv.rope_cache_write_fp4(e[:, :1], e[:, 1:2], e[:, 2:], pos[:0], rope, kd, vd, torch.empty(0, dtype=torch.int64).cuda()).shape == (0, 1, 64)


# ---------------------------------------------------------------------------------------------
# read
# ---------------------------------------------------------------------------------------------
LENS = [1, 15, 16, 17, 0, 100, 513, 31]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,hkv", [(128, 3), (64, 8), (256, 1), (16, 2), (80, 5), (240, 1)])
@pytest.mark.parametrize("window", [0, 1, 18, 16, 40])
def test_read_matches(pkv, D, hkv, dtype, window):
    p = F.Batch(D + hkv, LENS, hkv, D)
    dev = p.device()
    width = p.tables.shape[1]
    first = [max(0, n - window) // 16 if window else 0 for n in LENS]
    for b, f in enumerate(first):                                    # released blocks before the window
        dev[2][b, :f] = -1
    ko = torch.full((len(LENS) * width, hkv, 16, D), 7.0, dtype=dtype, device="cuda")
    vo, status = ko.clone(), _status()
    k, v = pkv.cache_read_fp4(*dev, window=window, key_out=ko, value_out=vo, status=status)
    assert k is ko and v is vo and int(status.item()) == 0
    for pool, out in ((p.kc, ko), (p.vc, vo)):
        want = np.full((len(LENS), width, hkv, 16, D), 7.0)
        val = F.unpack(pool)[2]
        for b, n in enumerate(LENS):
            for j in range(first[b], -(-n // 16)):
                want[b, j] = val[p.tables[b, j]]
                want[b, j, :, max(0, n - 16 * j):] = 0
        assert np.array_equal(out.double().cpu().numpy().reshape(want.shape), want)


def test_read_shapes_and_bounds(pkv):
    p = F.Batch(4, [40, 3, 70], 2, 64)
    dev = p.device()
    k, v = pkv.cache_read_fp4(*dev)
    assert k.shape == (15, 2, 16, 64) and k.dtype == v.dtype == torch.bfloat16
    k, v = pkv.cache_read_fp4(*dev, dtype=torch.float32, max_context_len=33)
    assert k.shape == (9, 2, 16, 64) and k.dtype == torch.float32
    # contexts of 40 and 70 are cut to three blocks
    status = _status()
    ko = torch.zeros(9, 2, 16, 64, device="cuda")
    vo = torch.zeros_like(ko)
    pkv.cache_read_fp4(*dev, max_context_len=33, key_out=ko, value_out=vo, status=status)
    assert int(status.item()) == 2
    val = F.unpack(p.kc)[2]
    assert np.array_equal(ko[6:].double().cpu().numpy(), val[p.tables[2, :3]])
    assert pkv.cache_read_fp4(*dev, max_context_len=1000)[0].shape[0] == 15
    # an entry out of range is read as block 0; lengths out of range are clamped
    bad = dev[2].clone()
    bad[0, 0], bad[2, 1] = p.blocks, -5
    lens = torch.tensor([16, -3, 32], dtype=torch.int32, device="cuda")
    status.zero_()
    ko.zero_()
    pkv.cache_read_fp4(dev[0], dev[1], bad, lens, max_context_len=48, key_out=ko, value_out=vo, status=status)
    assert int(status.item()) == 3
    first = F.unpack(p.kc)[2][0]
    assert np.array_equal(ko[0].double().cpu().numpy(), first, equal_nan=True)
    assert np.array_equal(ko[7].double().cpu().numpy(), first, equal_nan=True) and (ko[3:6] == 0).all()
    # nothing to read
    assert pkv.cache_read_fp4(dev[0], dev[1], dev[2][:0], dev[3][:0])[0].shape[0] == 0
    assert pkv.cache_read_fp4(dev[0], dev[1], dev[2][:, :0].contiguous(), dev[3] * 0)[0].shape[0] == 0


# ---------------------------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------------------------
DLENS = [1, 15, 16, 17, 0, 100, 513, 1100, 31]


@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 8), (128, 8, 4), (128, 6, 2), (128, 8, 2), (128, 5, 1), (128, 12, 2), (128, 7, 1),
                                      (128, 16, 2), (128, 11, 1), (128, 24, 2), (128, 16, 1), (64, 8, 2), (64, 5, 1), (64, 3, 3),
                                      (256, 4, 2), (256, 8, 1), (256, 2, 2)])
@pytest.mark.parametrize("partition", [0, 64, 16384])
def test_decode_matches(pkv, D, hq, hkv, partition):
    p = F.Batch(hq * 10 + hkv + D, DLENS, hkv, D)
    q, status = p.query(len(DLENS), hq), _status()
    out = pkv.decode_fp4(q.cuda(), *p.device(), partition_size=partition, status=status)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(DLENS)])
    F.check(out, ref, bound, f"{D} {hq}/{hkv} P={partition}")
    assert (out[4] == 0).all() and int(status.item()) == 0


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 513, 5000])
@pytest.mark.parametrize("D,hq,hkv,partition", [(128, 8, 8, 0), (128, 16, 2, 0), (64, 8, 2, 32), (256, 4, 1, 0)])
def test_decode_window(pkv, window, D, hq, hkv, partition):
    p = F.Batch(window, DLENS, hkv, D)
    q, dev = p.query(len(DLENS), hq), p.device()
    for b, n in enumerate(DLENS):                                    # released blocks before the window
        dev[2][b, :max(0, n - window) // 16] = -1
    status = _status()
    out = pkv.decode_fp4(q.cuda(), *dev, window=window, partition_size=partition, status=status)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(DLENS)], window=window)
    F.check(out, ref, bound, f"W={window}")
    assert int(status.item()) == 0


@pytest.mark.parametrize("seqs,hq,hkv,longest,width", [(1, 8, 2, 20000, None), (2, 4, 4, 3000, 2000), (40, 8, 8, 300, None),
                                                       (200, 8, 8, 60, None), (64, 16, 2, 700, 900), (3, 32, 32, 900, None)])
def test_decode_cuts(pkv, seqs, hq, hkv, longest, width):
    """Clusters, parts with a merge, one-warp CTAs, tables wider than the contexts."""
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, longest + 1, seqs)
    lens[0] = longest
    p = F.Batch(seqs, lens, hkv, 128, width=width)
    q = p.query(seqs, hq)
    out = pkv.decode_fp4(q.cuda(), *p.device())
    ref, bound = p.reference(q.double().numpy(), [(b, int(n) - 1) for b, n in enumerate(lens)])
    F.check(out, ref, bound, f"{seqs}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_values_of_any_size(pkv, D):
    """Keys and values from the smallest scales to the largest, large scores, rows of zeros."""
    lens = [500, 500, 500, 40]
    p = F.Batch(3, lens, 2, D, poison=False)
    x = torch.randn(p.blocks, 2, 16, D, generator=p.g, dtype=torch.float64)
    x *= torch.exp2(torch.randint(-18, 14, x.shape[:3], generator=p.g).double())[..., None]
    x = x.clamp(-61440, 61440)
    x[p.tables[3, 0]] = 0
    p.vc = F.pack(*F.encode(x.numpy()))
    q = p.query(4, 6)
    q[1] *= 2.0 ** -20
    q[2, 0] = 0
    out = pkv.decode_fp4(q.cuda(), *p.device())
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(lens)])
    F.check(out, ref, bound)
    # large scores: one position takes nearly all of the weight, references rise often
    out = pkv.decode_fp4(q.cuda(), *p.device(), scale=4.0)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(lens)], scale=4.0)
    # scores of up to 4 |q| |k| of f32 sums: 2^-22 of the sum of magnitudes moves a weight by as much
    kv = F.unpack(p.kc)[2]
    size = 4.0 * np.abs(q.double().numpy()).sum(-1).max() * np.abs(kv).max() * 2.0 ** -22
    F.check(out, ref, bound + 2 * size * np.abs(F.unpack(p.vc)[2]).max())


@pytest.mark.parametrize("seqs,hq,hkv,D,longest,window,plan", [
    (100, 8, 8, 128, 480, 0, False), (256, 4, 4, 128, 576, 0, False), (255, 8, 4, 128, 592, 0, True), (131, 16, 8, 64, 624, 0, True),
    (77, 8, 8, 256, 656, 0, False), (200, 16, 4, 128, 800, 480, False), (33, 32, 32, 128, 608, 0, False)])
def test_decode_longest_first(pkv, seqs, hq, hkv, D, longest, window, plan):
    """More than four CTAs an SM (two with heads of 256), a part each, and long for their number: CTAs take the longest
    sequences first.  Ragged ones, equal ones, empty ones and lengths out of range, each computed once."""
    assert pkv.decode_fp4_workspace_bytes(seqs, hq, hkv, D, longest // 16, window=window) == 0
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, longest + 1, seqs)
    lens[5:25] = 48                                                  # of one length
    lens[[2, 3, 30]] = 0
    lens[[0, 31]] = longest
    p = F.Batch(seqs, lens, hkv, D, width=longest // 16)
    kc, vc, tables, given = p.device()
    given[0], given[2], given[31] = longest + 1, -7, 1 << 30         # clamped to what they are
    for b, n in enumerate(lens):
        if window:
            tables[b, :max(0, n - window) // 16] = -1                # released blocks before the window
    brings = [b for b in range(seqs) if not plan or b % 5 != 1]
    q = p.query(len(brings) + 3, hq)
    start = np.cumsum([0] + [int(b in brings) for b in range(seqs)])
    status, out = _status(), torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    if plan:
        pkv.decode_fp4(q.cuda(), kc, vc, tables, given, query_start=torch.tensor(start, dtype=torch.int32, device="cuda"), window=window,
                       out=out, status=status)
    else:
        pkv.decode_fp4(q[:seqs].cuda(), kc, vc, tables, given, window=window, out=out[:seqs], status=status)
    ref, bound = p.reference(q[:len(brings)].double().numpy(), [(b, int(lens[b]) - 1) for b in brings], window=window)
    F.check(out[:len(brings)], ref, bound, f"{seqs}")
    assert (out[len(brings):] == 5).all() and int(status.item()) == 2


def _growing(p, size):
    """Keys of p grow along the contexts: those of position i of sequence b by size(b, i)."""
    x = torch.randn(p.blocks, p.hkv, 16, p.dim, generator=p.g, dtype=torch.float64)
    for b, n in enumerate(p.lens):
        for i in range(int(n)):
            x[p.tables[b, i // 16], :, i % 16] *= size(b, i)
    p.kc = F.pack(*F.encode(x.numpy()))
    p.scales(p.kc)[torch.from_numpy(~p.live)[:, None].expand(-1, p.hkv, -1)] = 0xFF


def _large_scores(p, q, rows, window=0, floor=1.0):
    """Batch.reference where scores are large: what f32 sums of a score change a weight by comes on top.

    Products are exact; each of D / 16 steps of 16 products adds at most 2^-22 of the sum of magnitudes A, and three
    roundings of the scaled score 3 times 2^-24 of it: a score is off by e = (D 2^-26 + 2^-22) scale A.  A weight
    p is then off by a factor of 1 + d, d = exp(e) - 1, and the output by at most sum p d |v - out| / (1 - sum p d)."""
    out, bound = p.reference(q, rows, window=window, floor=floor)
    group, scale = q.shape[1] // p.hkv, p.dim ** -0.5
    kv, vv = F.unpack(p.kc)[2], F.unpack(p.vc)[2]
    for i, (b, last) in enumerate(rows):
        pos = np.arange(max(0, last + 1 - window) if window else 0, last + 1)
        blk, off = p.tables[b][pos // 16], pos % 16
        for h in range(p.hkv):
            j = slice(h * group, (h + 1) * group)
            k, v = kv[blk, h, off], vv[blk, h, off]
            x = q[i, j] @ k.T * scale
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            d = np.expm1((p.dim * 2.0 ** -26 + 2.0 ** -22) * scale * (np.abs(q[i, j]) @ np.abs(k).T))
            far = np.einsum("gp,gpd->gd", w * d, np.abs(v[None] - out[i, j][:, None]))
            bound[i, j] += far / (1 - (w * d).sum(-1, keepdims=True))
    return out, bound


GROWTH = {"rising": lambda b, i: 0.5 + 24 * i / 700, "late": lambda b, i: 24.0 if i > 600 else 0.5,
          "halves": lambda b, i: (0.5 + 24 * i / 700) if (i // 64 + b) % 2 else 0.5, "falling": lambda b, i: 24.5 - 24 * i / 700,
          "steps": lambda b, i: 2.0 ** (i // 128)}


@pytest.mark.parametrize("growth", GROWTH)
@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (128, 8, 1), (128, 2, 2), (256, 4, 2)])
@pytest.mark.parametrize("partition", [0, 64])
def test_decode_references_that_rise(pkv, growth, D, hq, hkv, partition):
    """Scores that leave the reference behind again and again along a context: every output element within
    what its own weights are off by."""
    lens = [700, 655, 300, 40]
    p = F.Batch(3, lens, hkv, D)
    _growing(p, GROWTH[growth])
    q = p.query(4, hq)
    out = pkv.decode_fp4(q.cuda(), *p.device(), partition_size=partition)
    F.check(out, *_large_scores(p, q.double().numpy(), [(b, n - 1) for b, n in enumerate(lens)]), growth)


def test_decode_nan(pkv):
    """A NaN that is attended reaches its row and no other; NaN and infinite scales elsewhere reach none."""
    p = F.Batch(9, [50, 50, 50], 1, 128)
    q = p.query(3, 4)
    t = p.tables
    p.scales(p.vc)[t[0, 1], 0, 3, 2] = 0xFF                          # elements 32 .. 47 of position 19
    p.scales(p.kc)[t[1, 0], 0, 7, 0] = 0xFF
    p.scales(p.kc)[t[2, 3], 0, 2:] = 0xF8                            # behind 50 positions: infinite
    p.scales(p.vc)[t[2, 3], 0, 2:] = 0xF8
    out = pkv.decode_fp4(q.cuda(), *p.device()).float().cpu()
    assert out[0, :, 32:48].isnan().all() and not out[0, :, :32].isnan().any() and not out[0, :, 48:].isnan().any()
    assert out[1].isnan().all() and not out[2].isnan().any()
    # the window leaves both behind
    out = pkv.decode_fp4(q.cuda(), *p.device(), window=30).float().cpu()
    assert not out.isnan().any()


def test_decode_status_and_bounds(pkv):
    p = F.Batch(2, [40, 40, 40], 2, 128)
    q, dev = p.query(3, 4), p.device()
    bad = dev[2].clone()
    bad[1, 1] = 1 << 30
    status = _status()
    good = pkv.decode_fp4(q.cuda(), *dev)
    out = pkv.decode_fp4(q.cuda(), dev[0], dev[1], bad, dev[3], status=status)
    assert int(status.item()) == 1 and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    status.zero_()
    lens = torch.tensor([40, -1, 49], dtype=torch.int32, device="cuda")
    out = pkv.decode_fp4(q.cuda(), dev[0], dev[1], dev[2], lens, status=status)
    assert int(status.item()) == 2 and torch.equal(out[0], good[0]) and (out[1] == 0).all()
    status.zero_()
    big = q.clone()
    big[1, 2, 5] = 65536.0                                           # beyond f16, not beyond a query
    out = pkv.decode_fp4(big.cuda(), *dev, status=status)
    assert int(status.item()) == 0 and torch.equal(out[0], good[0]) and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("partition", [0, 16])
def test_decode_rows_of_a_plan(pkv, partition):
    lens = [30, 0, 77, 200, 16]
    p = F.Batch(6, lens, 2, 128)
    q, dev, status = p.query(4, 6), p.device(), _status()
    start = torch.tensor([0, 1, 1, 2, 2, 3], dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    pkv.decode_fp4(q.cuda(), *dev, query_start=start, out=out, partition_size=partition, status=status)
    ref, bound = p.reference(q[:3].double().numpy(), [(0, 29), (2, 76), (4, 15)])
    F.check(out[:3], ref, bound)
    assert (out[3] == 5).all() and int(status.item()) == 0           # a row of no sequence
    for entries, flag in (([0, 1, 3, 3, 3, 4], 64), ([0, 1, 0, 1, 2, 9], 2), ([-1, 0, 0, 1, 1, 2], 2)):
        status.zero_()
        pkv.decode_fp4(q.cuda(), *dev, query_start=torch.tensor(entries, dtype=torch.int32, device="cuda"), out=out,
                       partition_size=partition, status=status)
        assert int(status.item()) & flag


def test_pools_past_four_gigabytes(pkv):
    """Blocks whose bytes begin past 2^32: written, read back and attended."""
    hkv, D = 16, 128
    blocks = (1 << 32) // (hkv * 9 * D) + 40
    kc = torch.zeros(blocks, hkv, 16, 9 * D // 16, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(32, 2 * hkv, D, generator=g).to(torch.bfloat16)
    table = torch.tensor([[blocks - 1, blocks - 30]], dtype=torch.int32)
    slots = (table[0].long()[:, None] * 16 + torch.arange(16)).flatten()
    pkv.rope_cache_write_fp4(None, x[:, :hkv].cuda(), x[:, hkv:].cuda(), None, None, kc, vc, slots.cuda())
    k, v = pkv.cache_read_fp4(kc, vc, table.cuda(), torch.tensor([32], dtype=torch.int32).cuda(), dtype=torch.float32)
    want = F.values_of(*F.encode(x.double().numpy()))
    want = want.reshape(2, 16, 2 * hkv, D).transpose(0, 2, 1, 3)
    assert np.array_equal(k.double().cpu().numpy(), want[:, :hkv]) and np.array_equal(v.double().cpu().numpy(), want[:, hkv:])
    q = torch.randn(1, hkv, D, generator=g).to(torch.bfloat16)
    out = pkv.decode_fp4(q.cuda(), kc, vc, table.cuda(), torch.tensor([32], dtype=torch.int32).cuda())
    p = torch.softmax(torch.einsum("hd,hpd->hp", q[0].double(), torch.from_numpy(want[:, :hkv].transpose(1, 0, 2, 3).reshape(hkv, 32, D))) * D ** -0.5, -1)
    vv = torch.from_numpy(want[:, hkv:].transpose(1, 0, 2, 3).reshape(hkv, 32, D))
    ref = torch.einsum("hp,hpd->hd", p, vv)
    mass = torch.einsum("hp,hpd->hd", p, vv.abs())
    err = (out[0].double().cpu() - ref).abs()
    assert (err <= (2.0 ** -11 + 2.0 ** -15) * 2 * mass + 2.0 ** -8 * ref.abs()).all()


# ---------------------------------------------------------------------------------------------
# prefill
# ---------------------------------------------------------------------------------------------
def _rows(lens, new):
    return [(b, n - t + i) for b, (n, t) in enumerate(zip(lens, new)) for i in range(t)]


@pytest.mark.parametrize("hq,hkv", [(4, 4), (4, 2), (8, 2), (16, 2), (16, 1)])
@pytest.mark.parametrize("behind", [2, 4096], ids=["rows", "tiles"])     # of more than 4096 rows every chunk is tiles
@pytest.mark.parametrize("window", [0, 1, 37, 300])
def test_prefill_matches(pkv, hq, hkv, window, behind):
    lens, new = [1, 17, 130, 300, 64, 0, 33], [1, 17, 100, 3, 0, 0, 16]
    p = F.Batch(hq + window, lens, hkv, 128)
    dev = p.device()
    q, status = p.query(sum(new) + behind, hq), _status()
    assert _by_rows(pkv, 7, hq, hkv, 128, 19, len(q), 100, 300, window) == (behind == 2)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    if window:
        for b, (n, t) in enumerate(zip(lens, new)):
            dev[2][b, :max(0, n - t + 1 - window) // 16] = -1
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    got = pkv.prefill_fp4(q.cuda(), *dev, start, window=window, out=out, status=status)
    assert got is out and int(status.item()) == 0
    n = sum(new)
    ref, bound = p.reference(q[:n].double().numpy(), _rows(lens, new), window=window, floor=4.0)
    F.check(out[:n], ref, bound, f"{hq}/{hkv} W={window}")
    assert (out[n:] == 5).all()
    # blocks of the longest context only
    again = pkv.prefill_fp4(q.cuda(), *dev, start, 100, window=window, max_context_len=300,
                            workspace=torch.full((pkv.prefill_fp4_workspace_bytes(7, hq, hkv, 128, 19, n + behind, 100, 300, window),), 0xFF,
                                                 dtype=torch.uint8, device="cuda"))
    assert torch.equal(again[:n], out[:n])


@pytest.mark.parametrize("behind", [0, 4096], ids=["rows", "tiles"])
def test_prefill_refuses_rows_on_the_device(pkv, behind):
    """Sequences whose rows leave the query, or whose context is too long, are left out and flagged."""
    lens, new = [40, 40, 40], [10, 10, 10]
    p = F.Batch(1, lens, 1, 128)
    q, dev, status = p.query(30, 4), p.device(), _status()
    ref, bound = p.reference(q.double().numpy(), _rows(lens, new), floor=4.0)
    q = torch.cat([q, p.query(behind, 4)])
    # (in the last one rows 5 .. 9 are both the first's and the third's)
    for start, ok, rows in (([0, 10, 20, 31 + behind], [0, 1], 10), ([-1, 10, 20, 30], [1, 2], 10), ([0, 10, 5, 15], [0], 5)):
        status.zero_()
        out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        pkv.prefill_fp4(q.cuda(), *dev, torch.tensor(start, dtype=torch.int32, device="cuda"), 10, out=out, status=status)
        assert int(status.item()) & 2
        for b in ok:
            at = slice(10 * b, 10 * b + rows)
            F.check(out[at], ref[at], bound[at], f"{start} {b}")
    status.zero_()
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    pkv.prefill_fp4(q.cuda(), *dev, torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda"), 10, max_context_len=30,
                    out=out, status=status)
    assert int(status.item()) == 2 and (out == 5).all()


def _by_rows(pkv, *args):
    """Whether these sizes are computed a row at a time: then no block is staged."""
    return pkv.prefill_fp4_workspace_bytes(*args) < args[0] * args[4] * args[2] * 2 * 16 * 128 * 2


@pytest.mark.parametrize("hq,hkv", [(16, 2), (8, 2), (4, 2), (2, 2), (16, 1)])
@pytest.mark.parametrize("window", [0, 1, 40, 1000])
def test_prefill_of_few_rows(pkv, hq, hkv, window):
    """Short chunks on long contexts, as rows of a decode: against the formula and against tiles."""
    lens, new = [2000, 5, 0, 777, 16, 1600], [3, 5, 0, 1, 4, 8]
    p = F.Batch(hq + window, lens, hkv, 128)
    n, dev, status = sum(new), p.device(), _status()
    assert _by_rows(pkv, 6, hq, hkv, 128, p.tables.shape[1], n + 3, 8, None, window)
    if window:
        for b, (m, t) in enumerate(zip(lens, new)):
            dev[2][b, :max(0, m - t + 1 - window) // 16] = -1
    q = p.query(n + 4096, hq)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    out = torch.full((n + 3, hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    few = q[:n + 3].cuda()
    pkv.prefill_fp4(few, *dev, start, 8, window=window, out=out, status=status)
    assert int(status.item()) == 0 and (out[n:] == 5).all()
    ref, bound = p.reference(q[:n].double().numpy(), _rows(lens, new), window=window, floor=4.0)
    F.check(out[:n], ref, bound, f"{hq}/{hkv} W={window} rows")
    tiles = pkv.prefill_fp4(q.cuda(), *dev, start, 8, window=window)
    F.check(tiles[:n], ref, bound, f"{hq}/{hkv} W={window} tiles")

    # captured, replayed, with other lengths behind the same addresses
    work = torch.full((pkv.prefill_fp4_workspace_bytes(6, hq, hkv, 128, p.tables.shape[1], n + 3, 8, None, window),), 0xFF,
                      dtype=torch.uint8, device="cuda")
    graph, held = torch.cuda.CUDAGraph(), torch.zeros_like(out)
    with torch.cuda.graph(graph):
        pkv.prefill_fp4(few, *dev, start, 8, window=window, out=held, workspace=work)
    for _ in range(2):
        held.fill_(5)
        work.fill_(0xFF)
        graph.replay()
        assert torch.equal(held, out)
    dev[3][0] = 1990                                                 # rows 0 .. 2 end at 1990 now
    dev[2][0, :] = dev[2][0, :].clamp(min=0)                         # (the window reaches back further)
    held.fill_(5)
    graph.replay()
    if not window:
        ref, bound = p.reference(q[:3].double().numpy(), [(0, m) for m in (1987, 1988, 1989)], floor=4.0)
        F.check(held[:3], ref, bound, "shorter")
    assert torch.equal(held[3:], out[3:])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (8, 1)])
def test_prefill_of_few_rows_in_any_order(pkv, hq, hkv):
    """Sequences whose rows do not lie in the sequences' order, one of which is refused; and more
    sequences than a pass of the kernel that cuts the rows takes."""
    p = F.Batch(8, [600, 40, 90, 333], hkv, 128)
    q, dev, status = p.query(40, hq), p.device(), _status()
    start = torch.tensor([20, 33, 0, 17, 19], dtype=torch.int32, device="cuda")     # the second one falls
    assert _by_rows(pkv, 4, hq, hkv, 128, p.tables.shape[1], 40, 17)
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    pkv.prefill_fp4(q.cuda(), *dev, start, 17, out=out, status=status)
    assert int(status.item()) == 2
    rows = {20 + i: (0, 587 + i) for i in range(13)} | {i: (2, 73 + i) for i in range(17)} | {17 + i: (3, 331 + i) for i in range(2)}
    at = sorted(rows)
    ref, bound = p.reference(q[at].double().numpy(), [rows[i] for i in at], floor=4.0)
    F.check(out[at], ref, bound)
    assert (out[[i for i in range(40) if i not in rows]] == 5).all()

    lens = [1 + (7 * i) % 37 for i in range(1100)]
    new = [min(n, i % 4) for i, n in enumerate(lens)]
    p = F.Batch(9, lens, hkv, 128)
    n, dev = sum(new), p.device()
    q = p.query(n, hq)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    assert _by_rows(pkv, 1100, hq, hkv, 128, p.tables.shape[1], n, 3)
    out = pkv.prefill_fp4(q.cuda(), *dev, start, 3)
    ref, bound = p.reference(q.double().numpy(), _rows(lens, new), floor=4.0)
    F.check(out, ref, bound)


@pytest.mark.parametrize("power", [-60, 20, 40, 100])
def test_queries_of_any_magnitude(pkv, power):
    """A power of two taken from the scale and given to the query changes no bit, beyond f16's range too."""
    lens = [300, 33, 700]
    p = F.Batch(5, lens, 2, 128)
    dev, q, status = p.device(), p.query(12, 8).cuda(), _status()
    far = (q.float() * 2.0 ** power).to(torch.bfloat16)
    for f in (lambda x, scale: pkv.decode_fp4(x[:3], *dev, scale, status=status),
              lambda x, scale: pkv.prefill_fp4(x, *dev, start, 4, scale, status=status)):
        start = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device="cuda")
        assert torch.equal(f(far, 2.0 ** -(4 + power)), f(q, 2.0 ** -4))
    assert int(status.item()) == 0


def test_prefill_of_few_rows_longer_than_said(pkv):
    """Rows behind max_query_len are flagged and left as they were."""
    p = F.Batch(3, [900, 900], 2, 128)
    q, dev, status = p.query(12, 4), p.device(), _status()
    start = torch.tensor([0, 4, 12], dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    assert _by_rows(pkv, 2, 4, 2, 128, p.tables.shape[1], 12, 6)
    pkv.prefill_fp4(q.cuda(), *dev, start, 6, out=out, status=status)
    assert int(status.item()) == 64 and (out[10:] == 5).all()
    ref, bound = p.reference(q[:10].double().numpy(), _rows([900, 900], [4, 8])[:10], floor=4.0)
    F.check(out[:10], ref, bound)


def _in_parts(pkv, seqs, hq, hkv, width, rows, longest, window=0):
    """Whether these sizes are computed by rows whose contexts are cut into parts: partial results need room
    beside the chunks (16 bytes each) and their lengths (4)."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    heads = max(h for h in range(1, 9) if (hq // hkv) % h == 0)
    chunks = min(rows, rows // (8 // heads) + seqs)
    return pkv.prefill_fp4_workspace_bytes(seqs, hq, hkv, 128, width, rows, longest, None, window) > up(16 * chunks) + up(4 * chunks)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (4, 1), (8, 1), (16, 1), (16, 2), (4, 4)])
@pytest.mark.parametrize("lens,new,window", [
    ([6147], [5], 0), ([6144 + 8], [8], 0), ([6400], [2], 4500), ([6147], [5], 4500),       # (rows that end before the last part)
    ([6147, 1, 300, 6400, 5], [3, 2, 1, 4, 2], 0)])                                        # (the second one is refused)
def test_prefill_of_few_rows_in_parts(pkv, hq, hkv, lens, new, window):
    """Chunks whose contexts are cut into parts: partial results of several rows in a CTA's columns, merged."""
    p = F.Batch(hq + len(lens), lens, hkv, 128, width=400)
    n, dev, status = sum(new), p.device(), _status()
    assert _by_rows(pkv, len(lens), hq, hkv, 128, 400, n, max(new), None, window)
    assert _in_parts(pkv, len(lens), hq, hkv, 400, n, max(new), window) == (hq < 16 or new != [8])       # (those: clusters)
    if window:
        for b, (m, t) in enumerate(zip(lens, new)):
            dev[2][b, :max(0, m - t + 1 - window) // 16] = -1
    q = p.query(n, hq)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    rows, ok = _rows(lens, new), [i for b, t in enumerate(new) for i in range(sum(new[:b]), sum(new[:b]) + t) if t <= lens[b]]
    ref, bound = p.reference(q[ok].double().numpy(), [rows[i] for i in ok], window=window, floor=4.0)
    need = pkv.prefill_fp4_workspace_bytes(len(lens), hq, hkv, 128, 400, n, max(new), None, window)
    for fill in (0xFF, 0):                                           # what an earlier call left there does not matter
        work = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        pkv.prefill_fp4(q.cuda(), *dev, start, max(new), window=window, out=out, workspace=work, status=status)
        F.check(out[ok], ref, bound, f"{hq}/{hkv} {lens} W={window}")
        assert (out[[i for i in range(n) if i not in ok]] == 5).all()
    assert int(status.item()) == (2 if len(ok) < n else 0)


@pytest.mark.parametrize("hq,hkv,seqs", [(64, 8, 64), (32, 8, 64), (8, 8, 64), (16, 8, 90)])
def test_prefill_of_few_rows_longest_first(pkv, hq, hkv, seqs):
    """More chunks than fit the GPU at once, a part each: taken longest first, entries without a chunk among them."""
    rng = np.random.default_rng(hq)
    lens = rng.integers(4, 801, seqs).tolist()
    lens[0], lens[1], lens[2] = 800, 4, 0
    new = [min(n, 1 + int(rng.integers(0, 4))) for n in lens]
    p = F.Batch(hq, lens, hkv, 128, width=50)
    n, status = sum(new), _status()
    assert _by_rows(pkv, seqs, hq, hkv, 128, 50, n, 4) and not _in_parts(pkv, seqs, hq, hkv, 50, n, 4)
    q = p.query(n, hq)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    pkv.prefill_fp4(q.cuda(), *p.device(), start, 4, out=out, status=status)
    ref, bound = p.reference(q.double().numpy(), _rows(lens, new), floor=4.0)
    F.check(out, ref, bound, f"{hq}/{hkv}")
    assert int(status.item()) == 0


@pytest.mark.parametrize("growth", GROWTH)
@pytest.mark.parametrize("hq,hkv,window", [(4, 4, 0), (8, 2, 0), (16, 1, 0), (4, 4, 200), (8, 2, 100)])
@pytest.mark.parametrize("behind", [0, 4096], ids=["rows", "tiles"])
def test_prefill_references_that_rise(pkv, growth, hq, hkv, window, behind):
    """The same in prefill, in one half of a step's columns too and beside a window's end."""
    lens, new = [700, 300], [300 if behind else 30, 40 if behind else 5]
    p = F.Batch(window + hq, lens, hkv, 128)
    _growing(p, GROWTH[growth])
    n = sum(new)
    q = p.query(n + behind, hq)
    assert _by_rows(pkv, 2, hq, hkv, 128, p.tables.shape[1], len(q), max(new), None, window) == (behind == 0)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    out = pkv.prefill_fp4(q.cuda(), *p.device(), start, window=window)
    F.check(out[:n], *_large_scores(p, q[:n].double().numpy(), _rows(lens, new), window, floor=4.0), growth)


@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (16, 1)])
@pytest.mark.parametrize("window", [0, 150])
def test_prefill_nan(pkv, hq, hkv, window):
    """Tiles: a NaN key makes the rows that attend to it NaN and no other, a NaN value its elements of
    those rows (and perhaps of others of the chunk); another sequence's, head's or unit's nothing."""
    lens, new = [500, 333, 260], [300, 100, 260]
    p = F.Batch(hq, lens, hkv, 128)
    n, group, t = sum(new), hq // hkv, p.tables
    q = p.query(n + 4096, hq)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    ref, bound = p.reference(q[:n].double().numpy(), _rows(lens, new), window=window, floor=4.0)
    p.scales(p.kc)[t[0, 270 // 16], 0, 270 % 16, 3] = 0xFF           # position 270, seen by the rows from 70 on
    p.scales(p.vc)[t[1, 300 // 16], hkv - 1, 300 % 16, 5] = 0xFF     # elements 80 .. 95 of position 300
    out = pkv.prefill_fp4(q.cuda(), *p.device(), start, window=window)[:n].double().cpu().numpy()
    rows = np.array(_rows(lens, new))
    sees = (rows[:, 0] == 0) & (rows[:, 1] >= 270) & (rows[:, 1] < (270 + window if window else 10 ** 6))
    assert np.isnan(out[sees][:, :group]).all() and 100 < sees.sum() < 300
    reads = (rows[:, 0] == 1) & (rows[:, 1] >= 300) & (rows[:, 1] < (300 + window if window else 10 ** 6))
    assert np.isnan(out[reads][:, hq - group:, 80:96]).all() and reads.sum() == 33
    clean = np.ones(out.shape, bool)
    clean[sees, :group] = False
    clean[300:400, hq - group:, 80:96] = False
    assert not np.isnan(out[clean]).any()
    F.check(torch.from_numpy(np.where(clean, out, ref)), ref, bound)


# ---------------------------------------------------------------------------------------------
# blocks that move
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D,hkv", [(128, 2), (64, 1), (16, 1), (80, 3)])
def test_copy_and_swap(pkv, D, hkv):
    g = torch.Generator().manual_seed(D)
    kc, vc = F.pool(g, 9, hkv, D), F.pool(g, 9, hkv, D)
    kd, vd = kc.cuda(), vc.cuda()
    pkv.block_copy(kd, vd, torch.tensor([[2, 7], [0, 8]], dtype=torch.int32).cuda())
    for src, pool in ((kc, kd), (vc, vd)):
        want = src.clone()
        want[7], want[8] = src[2], src[0]
        assert torch.equal(pool.cpu(), want)
    ids = torch.tensor([3, 1], dtype=torch.int32).cuda()
    staging = pkv.swap_out(kd, vd, ids)
    torch.cuda.synchronize()
    assert torch.equal(staging[:, 0], kc[[3, 1]]) and torch.equal(staging[:, 1], vc[[3, 1]])
    back = torch.tensor([5, 6], dtype=torch.int32).cuda()
    pkv.swap_in(kd, vd, back, staging)
    assert torch.equal(kd[5:7].cpu(), kc[[3, 1]]) and torch.equal(vd[5:7].cpu(), vc[[3, 1]])
