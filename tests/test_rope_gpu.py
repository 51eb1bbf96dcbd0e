"""pa_rope_cache_write: rotary positions on queries and keys with the cache write, into f32, bf16
and block-scaled E4M3 pools, against 64-bit implementations."""
import numpy as np
import pytest
import torch

from tests import block8_ref as R

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


def _inputs(seed, T, Hq, Hkv, D, dtype, blocks, far=False):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g) * torch.exp2(torch.randn(T, Hq + 2 * Hkv, 1, generator=g))
    qkv = qkv.to(dtype)
    pos = torch.randint(0, 1 << 30 if far else 5000, (T,), generator=g, dtype=torch.int32)
    slots = torch.randperm(blocks * 16, generator=g)[:T]
    return g, qkv, pos, slots


def _close(got, ref, mass, a, dtype, what):
    err = np.abs(got.double().cpu().numpy() - ref)
    bound = a * TURN * mass + HALF_STEP[dtype] * (np.abs(ref) + a * TURN * mass)
    assert (err <= bound).all(), (what, float((err - bound).max()))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (128, 20), (64, 2), (256, 250), (96, 96), (80, 0), (8, 6)])
def test_rows_match(pkv, D, rot, dtype, interleaved):
    T, Hq, Hkv, blocks = 21, 5, 2, 4
    g, qkv, pos, slots = _inputs(D + rot, T, Hq, Hkv, D, dtype, blocks)
    slots[3] = -1
    rope = pkv.rotary_plan(rot, interleaved=interleaved)
    x = qkv.cuda()
    kc = torch.randn(blocks, Hkv, 16, D, generator=g).to(dtype)
    vc = torch.randn(blocks, Hkv, 16, D, generator=g).to(dtype)
    kd, vd = kc.cuda(), vc.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.rope_cache_write(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos.cuda(), rope, kd, vd, slots.cuda(),
                               status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    cos, sin = R.rotary_angles(pos.numpy(), rot)
    ref, mass = R.rotate(qkv.double().numpy(), cos, sin, interleaved)
    _close(out, ref[:, :Hq], mass[:, :Hq], 1.0, dtype, "query")
    want, wmass = kc.double().numpy(), np.zeros(kc.shape)
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s // 16, :, s % 16] = ref[i, Hq:Hq + Hkv]
            wmass[s // 16, :, s % 16] = mass[i, Hq:Hq + Hkv]
            vc[s // 16, :, s % 16] = qkv[i, Hq + Hkv:]
    _close(kd, want, wmass, 1.0, dtype, "keys")
    assert torch.equal(vd.cpu(), vc)
    # the same call in place on contiguous queries
    q = x[:, :Hq].contiguous()
    same = pkv.rope_cache_write(q, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos.cuda(), rope, kd, vd, slots.cuda(), query_out=q)
    assert same is q and torch.equal(q, out)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("by_parts", 8.0)])
def test_scaled_and_far_positions(pkv, scaling, factor):
    T, H, D = 40, 3, 128
    _, qkv, pos, slots = _inputs(5, T, H, 1, D, torch.float32, 8, far=True)
    pos[:4] = torch.tensor([0, 1, 2 ** 31 - 1, 131071], dtype=torch.int32)
    rope = pkv.rotary_plan(D, 500000.0, scaling=scaling, factor=factor)
    x = qkv.cuda()
    pool = torch.zeros(8, 1, 16, D, device="cuda")
    out = pkv.rope_cache_write(x[:, :H], x[:, H:H + 1], x[:, H + 1:], pos.cuda(), rope, pool, torch.zeros_like(pool), slots.cuda())
    # in whole turns, so that the reference's own angle is exact at far positions
    turns = [int(t) % (1 << 64) for t in rope.turns.cpu().tolist()]
    frac = np.array([[((int(p) * t) % (1 << 64)) / 2.0 ** 64 for t in turns] for p in pos.tolist()])
    a = rope.attention_factor
    near, _ = R.rotary_angles(np.ones(1), D, 500000.0, scaling, factor)
    assert np.allclose(near[0], a * np.cos(2 * np.pi * np.array(turns) / 2.0 ** 64), atol=1e-7)
    ref, mass = R.rotate(qkv.double().numpy(), a * np.cos(2 * np.pi * frac), a * np.sin(2 * np.pi * frac), False)
    _close(out, ref[:, :H], mass[:, :H], a, torch.float32, scaling)


def _chunks(rng, seqs, longest, spare=2):
    """Slots of chunks that begin anywhere in a block; blocks in random order."""
    lens = rng.integers(0, 40, seqs)
    new = rng.integers(1, longest + 1, seqs)
    first = lens // 16
    need = -(-(lens + new) // 16) - first
    perm = rng.permutation(int(need.sum()) + spare)
    slots, pos, at = [], [], 0
    for b in range(seqs):
        for p in range(lens[b], lens[b] + new[b]):
            slots.append(int(perm[at + p // 16 - first[b]]) * 16 + p % 16)
            pos.append(p)
        at += need[b]
    return np.array(slots, np.int64), np.array(pos, np.int32), perm.size


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 96, True), (64, 50, False), (256, 256, False), (16, 16, False)])
@pytest.mark.parametrize("seqs,longest", [(1, 1), (5, 1), (4, 70), (40, 3)])
def test_block_scaled_write(pkv, seqs, longest, D, rot, interleaved, dtype):
    rng = np.random.default_rng(seqs * 1000 + longest + D)
    slots, pos, blocks = _chunks(rng, seqs, longest)
    T, Hq, Hkv = slots.size, 2, 3
    g, qkv, _, _ = _inputs(seqs + D, T, Hq, Hkv, D, dtype, blocks + T)
    kc, ks = R.pools(g, blocks, Hkv, D)
    vc, vs = R.pools(g, blocks, Hkv, D)
    qkv[T // 2, Hq:] = 0                                     # an all-zero row
    if T > 3:
        slots[T - 2] = -1
    x, d = qkv.cuda(), lambda t: t.cuda()  # noqa: E731
    kd, ksd, vd, vsd = d(kc), d(ks), d(vc), d(vs)
    rope = pkv.rotary_plan(rot, interleaved=interleaved)
    out = pkv.rope_cache_write(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], torch.from_numpy(pos).cuda(), rope,
                               kd, vd, torch.from_numpy(slots).cuda(), k_scales=ksd, v_scales=vsd)
    torch.cuda.synchronize()
    cos, sin = R.rotary_angles(pos, rot)
    ref, mass = R.rotate(qkv.double().numpy(), cos, sin, interleaved)
    _close(out, ref[:, :Hq], mass[:, :Hq], 1.0, dtype, "query")
    kv, vv = R.decode_codes(kc), R.decode_codes(vc)
    kss, vss = ks.double().numpy().copy(), vs.double().numpy().copy()
    R.write_blocks(qkv[:, Hq + Hkv:].double().numpy(), slots, vv, vss)
    assert np.array_equal(vsd.cpu().double().numpy(), vss)
    assert np.array_equal(R.decode_codes(vd), vv)            # values are not turned: every code is the same
    R.write_blocks(ref[:, Hq:Hq + Hkv], slots, kv, kss)
    assert np.array_equal(ksd.cpu().double().numpy(), kss)
    got = R.decode_codes(kd)
    # a key next to the border of two codes may take either: one step of the code, in few places
    step = 2.0 ** (np.clip(np.floor(np.log2(np.maximum(np.abs(kv), 2.0 ** -9))), -6, 8) - 3)
    assert (np.abs(got - kv) <= step * 1.001).all() and (got != kv).mean() < 1e-3


def test_block_scaled_write_grows_a_block_token_by_token(pkv):
    """Sixteen single-token writes with growing magnitudes: the scale grows, earlier rows follow."""
    D, H = 128, 2
    g = torch.Generator().manual_seed(8)
    rows = (torch.randn(16, H, D, generator=g) * 2.0 ** torch.arange(-8, 8)[:, None, None]).to(torch.bfloat16)
    kc = torch.full((3, H, 16, D), 0x7F, dtype=torch.uint8, device="cuda")      # stale codes, NaN among them
    vc, ks, vs = kc.clone(), torch.full((3, H), 1e9, device="cuda"), torch.full((3, H), 1e9, device="cuda")
    kv, kss = R.decode_codes(kc), ks.double().cpu().numpy()
    for i in range(16):
        pkv.rope_cache_write(None, rows[i:i + 1].cuda(), rows[i:i + 1].cuda(), None, None, kc, vc,
                             torch.tensor([16 + i], device="cuda"), k_scales=ks, v_scales=vs)
        R.write_blocks(rows[i:i + 1].double().numpy(), [16 + i], kv, kss)
        assert np.array_equal(R.decode_codes(kc)[1, :, :i + 1], kv[1, :, :i + 1])
        assert np.array_equal(ks.double().cpu().numpy(), kss) and torch.equal(ks, vs) and torch.equal(kc, vc)
    assert (kc[0] == 0x7F).all() and (kc[2] == 0x7F).all()


def test_block_scaled_write_special_values(pkv):
    from paged_kv_cache_100_gb300 import _lib
    D, H = 128, 1
    rows = torch.zeros(4, H, D, dtype=torch.bfloat16)
    rows[0, 0, :3] = torch.tensor([float("nan"), 1.0, -2.0])
    rows[1, 0, :2] = torch.tensor([float("inf"), 5.0])
    rows[2, 0, :2] = torch.tensor([1e-30, 3.0e-30])
    rows[3, 0, :2] = torch.tensor([448.0, -448.0])
    kc = torch.zeros(4, H, 16, D, dtype=torch.uint8, device="cuda")
    vc, ks, vs = kc.clone(), torch.zeros(4, H, device="cuda"), torch.zeros(4, H, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 16, 32, 48], device="cuda")
    pkv.rope_cache_write(None, rows.cuda(), rows.cuda(), None, None, kc, vc, slots, k_scales=ks, v_scales=vs, status=status)
    v = R.decode_codes(kc)[:, 0, 0]
    s = ks.cpu().double().numpy()[:, 0]
    assert np.isnan(v[0, 0]) and (v[0, 1:3] * s[0]).tolist() == [1.0, -2.0] and s[0] == 2.0 ** -7
    assert v[1, 0] == 448 and s[1] == 2.0 ** 31 and int(status.item()) == _lib.PA_DEV_RANGE
    assert (v[2] == 0).all() and s[2] == 2.0 ** -32
    assert v[3, 0] == 448 and v[3, 1] == -448 and s[3] == 1.0


def test_block_scaled_write_duplicates_holes_and_spread_blocks(pkv):
    """Holes and repeated slots inside a block's run, a block whose entries lie too far apart, a
    slot past the pool."""
    from paged_kv_cache_100_gb300 import _lib
    D, H, T = 128, 2, 45
    g = torch.Generator().manual_seed(2)
    rows = torch.randn(T, H, D, generator=g).to(torch.bfloat16)
    slots = np.full(T, -1, np.int64)
    slots[[0, 2, 5, 9]] = [20, 22, 21, 22]                   # block 1: offsets 4, 6, 5, and 6 again
    slots[[3, 40]] = [48, 49]                                # block 3: 37 entries apart
    slots[7] = 4 * 16 + 5                                    # past the pool
    kc, ks = R.pools(g, 4, H, D)
    kd, ksd = kc.cuda(), ks.cuda()
    vd, vsd = kc.cuda(), ks.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.rope_cache_write(None, rows.cuda(), rows.cuda(), None, None, kd, vd, torch.from_numpy(slots).cuda(),
                         k_scales=ksd, v_scales=vsd, status=status)
    kv, kss = R.decode_codes(kc), ks.double().numpy().copy()
    slots[40] = -1                                           # dropped
    R.write_blocks(rows.double().numpy(), slots, kv, kss)
    assert np.array_equal(R.decode_codes(kd), kv) and np.array_equal(ksd.cpu().double().numpy(), kss)
    assert torch.equal(kd, vd) and torch.equal(ksd, vsd)
    assert int(status.item()) == _lib.PA_DEV_BAD_SLOT


def test_a_chosen_scale_is_kept_and_divided_by(pkv):
    """A part-filled block whose scale is no power of two and large enough keeps it."""
    D, H = 128, 1
    g = torch.Generator().manual_seed(4)
    rows = torch.randn(1, H, D, generator=g).to(torch.bfloat16)
    kc, ks = R.pools(g, 2, H, D)
    ks[1] = 0.1
    kd, ksd, vd, vsd = kc.cuda(), ks.cuda(), kc.cuda(), ks.cuda()
    pkv.rope_cache_write(None, rows.cuda(), rows.cuda(), None, None, kd, vd, torch.tensor([16 + 9], device="cuda"),
                         k_scales=ksd, v_scales=vsd)
    assert torch.equal(ksd.cpu(), ks)
    want = kc.clone()
    want[1, 0, 9] = (rows[0, 0].float() / torch.tensor(0.1)).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(kd.cpu(), want)


def test_large_batch_uses_many_tokens_per_block(pkv):
    """Enough tokens that one thread block takes several; checked against small calls."""
    rng = np.random.default_rng(1)
    slots, pos, blocks = _chunks(rng, 30, 600)
    T, Hq, Hkv, D = slots.size, 4, 2, 128
    g, qkv, _, _ = _inputs(3, T, Hq, Hkv, D, torch.bfloat16, blocks + T)
    x = qkv.cuda()
    rope = pkv.rotary_plan(D)
    kc, ks = R.pools(g, blocks, Hkv, D)
    a, b = [[t.cuda() for t in (kc, ks, kc, ks)] for _ in range(2)]
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda()
    run = lambda c, lo, hi: pkv.rope_cache_write(  # noqa: E731
        x[lo:hi, :Hq], x[lo:hi, Hq:Hq + Hkv], x[lo:hi, Hq + Hkv:], p[lo:hi], rope, c[0], c[2], s[lo:hi],
        k_scales=c[1], v_scales=c[3])
    whole = run(a, 0, T)
    ends = [0] + [i for i in range(1, T) if slots[i] // 16 != slots[i - 1] // 16] + [T]
    parts = [run(b, lo, hi) for lo, hi in zip(ends, ends[1:])]
    assert torch.equal(whole, torch.cat(parts))
    for u, v in zip(a, b):
        assert torch.equal(u, v)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot,interleaved,Hq,Hkv", [(256, 74, False, 1, 1), (128, 18, True, 3, 1), (64, 50, False, 2, 2),
                                                      (64, 64, True, 1, 1), (128, 128, False, 3, 1), (16, 2, False, 5, 3),
                                                      (128, 96, True, 0, 4), (64, 48, False, 0, 20), (256, 256, False, 1, 1)])
@pytest.mark.parametrize("seqs,longest", [(2, 700), (6, 520), (130, 40), (40, 300), (60, 900)])
def test_large_batches_of_any_shape(pkv, seqs, longest, D, rot, interleaved, Hq, Hkv, dtype, codes):
    """Calls large enough that thread blocks take 2, 4, 8, 16 and 64 tokens' blocks (and several tokens' rows),
    in every kind of row, against calls of one sequence or part of one."""
    rng = np.random.default_rng(seqs + D + rot)
    slots, pos, blocks = _chunks(rng, seqs, longest)
    T = slots.size
    g, qkv, fk, fv = _inputs(seqs + rot, T, Hq, Hkv, D, dtype, blocks + T)
    x = qkv.cuda()
    rope = pkv.rotary_plan(rot, interleaved=interleaved)
    if codes:
        kc, ks = R.pools(g, blocks, Hkv, D)
        pool = (kc, ks, kc, ks)
    else:
        kc = torch.zeros(blocks, Hkv, 16, D, dtype=dtype)
        pool = (kc, None, kc, None)
    a, b = [[None if t is None else t.cuda() for t in pool] for _ in range(2)]
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run = lambda c, lo, hi: pkv.rope_cache_write(  # noqa: E731
        x[lo:hi, :Hq] if Hq else None, x[lo:hi, Hq:Hq + Hkv], x[lo:hi, Hq + Hkv:], p[lo:hi], rope, c[0], c[2], s[lo:hi],
        k_scales=c[1], v_scales=c[3], status=status)
    whole = run(a, 0, T)
    ends = [0]
    for i in range(1, T):
        if slots[i] // 16 != slots[i - 1] // 16 and i - ends[-1] > 150:
            ends.append(i)
    parts = [run(b, lo, hi) for lo, hi in zip(ends, ends[1:] + [T])]
    if Hq:
        assert torch.equal(whole, torch.cat(parts))
    for u, v in zip(a, b):
        assert u is None or torch.equal(u, v)
    assert int(status.item()) == 0


def test_tiles_shared_by_thread_blocks(pkv):
    """Many KV heads and several blocks begun per thread block: the thread blocks that share a tile's
    (block, head) pairs take each pair once, in every run."""
    rng = np.random.default_rng(3)
    slots, pos, blocks = _chunks(rng, 110, 11)
    T, Hkv, D = slots.size, 17, 64
    assert T >= 616                                          # two tokens a thread block
    g, qkv, _, _ = _inputs(5, T, 0, Hkv, D, torch.float32, blocks + T)
    x = qkv.cuda()
    rope = pkv.rotary_plan(D, interleaved=True)
    kc, ks = R.pools(g, blocks, Hkv, D)
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda()
    run = lambda c, lo, hi: pkv.rope_cache_write(  # noqa: E731
        None, x[lo:hi, :Hkv], x[lo:hi, Hkv:], p[lo:hi], rope, c[0], c[2], s[lo:hi], k_scales=c[1], v_scales=c[3])
    fresh = lambda: [t.cuda() for t in (kc, ks, kc, ks)]  # noqa: E731
    want = fresh()
    ends = [0] + [i for i in range(1, T) if slots[i] // 16 != slots[i - 1] // 16] + [T]
    for lo, hi in zip(ends, ends[1:]):
        run(want, lo, hi)
    for _ in range(30):
        got = fresh()
        run(got, 0, T)
        for u, v in zip(got, want):
            assert torch.equal(u, v)


def _groups(slots, limit):
    """The slots of a call whose tokens a block-scaled write stores, and the blocks that it does not answer for.
    Tokens of a block led by one entry are those among the 32 from it on; an entry 32 to 62 behind another of its
    block is dropped; groups farther apart race."""
    slots, by_block = np.asarray(slots), {}
    keep = np.full(slots.shape, -1, np.int64)
    for i, s in enumerate(slots):
        if 0 <= s < limit:
            by_block.setdefault(int(s) // 16, []).append(i)
    racing = []
    for blk, entries in by_block.items():
        keep[[i for i in entries if i - entries[0] < 32]] = slots[[i for i in entries if i - entries[0] < 32]]
        if max(np.diff(entries), default=0) > 62:
            racing.append(blk)
    return keep, racing


def _spread(rng, kind, n, blocks):
    if kind == "steps":                                      # token by token over 64 sequences
        return np.concatenate([np.arange(64) * 160 + 5 + t for t in range(n // 64)])
    if kind == "twice":                                      # a chunk, other tokens, the same chunk
        return np.concatenate([np.arange(7, n // 3), np.full(n // 3, -1), np.arange(7, n // 3)])
    parts = []
    while sum(map(len, parts)) < n:                          # whole blocks, pieces and gaps
        blk = int(rng.integers(0, blocks)) * 16
        x = rng.random()
        if x < 0.4:
            parts.append(blk + np.arange(16))
        elif x < 0.8:
            parts.append(blk + rng.integers(0, 16, int(rng.integers(1, 12))))
        else:
            parts.append(np.full(int(rng.integers(1, 90)), -1))
    return np.concatenate(parts)[:n]


@pytest.mark.parametrize("hkv", [1, 9])
@pytest.mark.parametrize("kind,n,blocks", [("steps", 640, 700), ("steps", 2560, 700), ("twice", 300, 40), ("twice", 6000, 400),
                                           ("mixed", 150, 8), ("mixed", 900, 100), ("mixed", 5000, 700), ("mixed", 21000, 4000)])
def test_tokens_of_a_block_far_apart(pkv, kind, n, blocks, hkv):
    """Tokens of one block anywhere in the list: the call is flagged, and all other blocks are written as ever."""
    from paged_kv_cache_100_gb300 import _lib
    D = 32
    rng = np.random.default_rng(n + blocks)
    slots = _spread(rng, kind, n, blocks).astype(np.int64)
    T = slots.size
    g = torch.Generator().manual_seed(n)
    rows = (torch.randn(T, hkv, D, generator=g) * torch.exp2(2 * torch.randn(T, hkv, 1, generator=g))).to(torch.bfloat16)
    kc, ks = R.pools(g, blocks, hkv, D)
    kv, kss = R.decode_codes(kc), ks.double().numpy().copy()
    keep, racing = _groups(slots, blocks * 16)
    R.write_blocks(rows.double().numpy(), keep, kv, kss)
    fine = np.setdiff1d(np.arange(blocks), racing)
    assert len(fine) > 0
    kd, ksd, vd, vsd = kc.cuda(), ks.cuda(), kc.cuda(), ks.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.rope_cache_write(None, rows.cuda(), rows.cuda(), None, None, kd, vd, torch.from_numpy(slots).cuda(),
                         k_scales=ksd, v_scales=vsd, status=status)
    assert int(status.item()) == (_lib.PA_DEV_BAD_SLOT if racing or (keep != slots).any() else 0)
    for codes, scales in ((kd, ksd), (vd, vsd)):
        assert np.array_equal(scales.cpu().double().numpy()[fine], kss[fine])
        assert np.array_equal(R.decode_codes(codes)[fine], kv[fine])


@pytest.mark.parametrize("n,at,back", [(33, 32, 32), (64, 63, 63), (64, 63, 31), (1025, 1024, 1024), (1100, 1050, 30),
                                       (20000, 19999, 19999), (20000, 17000, 600), (20000, 16400, 20), (20000, 1023, 1000)])
def test_one_token_far_from_the_others_of_its_block(pkv, n, at, back):
    """A single entry whose block another one has, at every distance: flagged beyond the 32 entries."""
    from paged_kv_cache_100_gb300 import _lib
    slots = torch.arange(n, dtype=torch.int64) * 16          # a block for every token
    slots[at] = slots[at - back] + 3
    rows = torch.ones(n, 1, 16, dtype=torch.bfloat16, device="cuda")
    codes = [torch.zeros(n, 1, 16, 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(n, 1, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.rope_cache_write(None, rows, rows, None, None, *codes, slots.cuda(), k_scales=scales[0], v_scales=scales[1], status=status)
    assert int(status.item()) == (_lib.PA_DEV_BAD_SLOT if back >= 32 else 0)


def _exact_keys(rope, pos, x, interleaved):
    """Keys [tokens][heads][D] turned in float64 from the plan's own 64-bit frequencies, and |x0| + |x1| of each
    element's pair (times the attention factor)."""
    turns = [int(t) % (1 << 64) for t in rope.turns.cpu().tolist()]
    whole = [[(int(p) * t) % (1 << 64) for t in turns] for p in pos]
    ang = 2 * np.pi * np.array([[(f - (1 << 64) if f >> 63 else f) / 2.0 ** 64 for f in row] for row in whole]).reshape(len(pos), -1)
    a = rope.attention_factor
    y, mass = R.rotate(x, a * np.cos(ang), a * np.sin(ang), interleaved)
    return y, a * mass


def _check_codes(pkv, rope, pos, keys, interleaved, close, expect_scales=None):
    """Writes keys, a block for every 16 tokens, and requires the code of the f32 quotient of the exact key
    everywhere.  The reference itself is off by a few units of 2^-53 of the pair's magnitudes: where 2^-46
    of them moves the code, either is right (and those are next to none).  `close`: so many elements at least
    lie where 2^-22 of the magnitudes, less than the error of 32-bit arithmetic, moves the code."""
    T, H, D = keys.shape
    blocks = -(-T // 16)
    codes = [torch.zeros(blocks, H, 16, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(blocks, H, device="cuda") for _ in range(2)]
    d = keys.cuda()
    pkv.rope_cache_write(None, d, d, torch.tensor(pos, dtype=torch.int32, device="cuda"), rope, *codes, torch.arange(T, device="cuda"),
                         k_scales=scales[0], v_scales=scales[1])
    y, mass = _exact_keys(rope, pos, keys.double().numpy(), interleaved)
    pad = np.zeros((blocks * 16 - T, H, D))
    by_block = lambda t: np.concatenate([t, pad]).reshape(blocks, 16, H, D).transpose(0, 2, 1, 3)  # noqa: E731
    y, mass = by_block(y), by_block(mass)
    s = scales[0].double().cpu().numpy()
    want = np.array([[R.block_scale(v) for v in row] for row in np.abs(y).max((2, 3))])
    assert np.array_equal(s, want)
    if expect_scales is not None:
        assert np.array_equal(s[:, 0], expect_scales)
    code = lambda v: torch.from_numpy((v / s[:, :, None, None]).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()  # noqa: E731
    got, low, high = codes[0].cpu().numpy(), code(y - 2.0 ** -46 * mass), code(y + 2.0 ** -46 * mass)
    assert (got == code(y)).mean() > 1 - 1e-5
    wrong = (got != low) & (got != high)
    assert not wrong.any(), (int(wrong.sum()), np.argwhere(wrong)[:3].tolist())
    assert (low != high).mean() < 1e-3
    assert (code(y - 2.0 ** -22 * mass) != code(y + 2.0 ** -22 * mass)).sum() >= close


SHAPES = [(128, 128, False), (128, 128, True), (128, 64, False), (128, 18, True), (64, 50, False), (256, 256, False), (16, 2, True),
          (80, 48, False)]


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("by_parts", 8.0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot,interleaved", SHAPES)
def test_codes_are_those_of_the_exact_keys(pkv, D, rot, interleaved, dtype, scaling, factor):
    """Half a million elements of each kind of row, some 70 of which lie where 32 bits do not tell their code."""
    g = torch.Generator().manual_seed(D + rot)
    T, H = (1 << 19) // (2 * D) + 5, 2
    keys = (torch.randn(T, H, D, generator=g) * torch.exp2(torch.randn(T, H, 1, generator=g))).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).tolist()
    _check_codes(pkv, pkv.rotary_plan(rot, 500000.0, interleaved=interleaved, scaling=scaling, factor=factor), pos, keys, interleaved, 1)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("by_parts", 8.0)])
@pytest.mark.parametrize("D,rot,interleaved", SHAPES)
def test_codes_beside_the_borders_of_codes(pkv, D, rot, interleaved, scaling, factor):
    """f32 rows whose first elements of pairs are solved for the border of two codes, one unit of the element
    below to one above it."""
    g = torch.Generator().manual_seed(7 * D + rot)
    T, half = 320, rot // 2
    rope = pkv.rotary_plan(rot, 500000.0, interleaved=interleaved, scaling=scaling, factor=factor)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).tolist()
    keys = torch.randn(T, 1, D, generator=g).numpy()
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    one = np.zeros((T, 1, D))
    one[..., first] = 1.0
    c = _exact_keys(rope, pos, one, interleaved)[0][..., first]
    one[..., first], one[..., second] = 0.0, 1.0
    s = -_exact_keys(rope, pos, one, interleaved)[0][..., first]
    # borders of codes: odd multiples of half a step, 16 to 31 quarters of it in each octave
    border = (torch.randint(8, 16, c.shape, generator=g).double().numpy() + 0.5) * 2.0 ** torch.randint(-8, -2, c.shape, generator=g).double().numpy()
    x0 = (border + keys[..., second] * s) / np.where(np.abs(c) < 0.05, 1.0, c)
    nudged = x0.astype(np.float32)
    nudge = torch.randint(-1, 2, c.shape, generator=g).numpy()
    for k in (-1, 1):
        nudged = np.where(nudge == k, np.nextafter(nudged, np.float32(k * np.inf)), nudged)
    keys[..., first] = nudged
    _check_codes(pkv, rope, pos, torch.from_numpy(keys), interleaved, T * half // 3)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("by_parts", 8.0)])
@pytest.mark.parametrize("D,rot,interleaved", SHAPES)
def test_scales_beside_their_borders(pkv, D, rot, interleaved, scaling, factor):
    """Blocks whose largest magnitude, a turned element, lies within a few units of 448 * 2^e, below and above."""
    g = torch.Generator().manual_seed(11 * D + rot)
    blocks, half = 96, rot // 2
    T = blocks * 16
    rope = pkv.rotary_plan(rot, 500000.0, interleaved=interleaved, scaling=scaling, factor=factor)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).tolist()
    keys = torch.randn(T, 1, D, generator=g).numpy()
    turns = [int(t) % (1 << 64) for t in rope.turns.cpu().tolist()]
    expect = np.zeros(blocks)
    for b in range(blocks):
        e = b % 7 - 4
        for _ in range(200):                                 # a token and a pair whose cosine is large
            t, i = 16 * b + int(torch.randint(0, 16, (1,), generator=g)), int(torch.randint(0, half, (1,), generator=g))
            ang = 2 * np.pi * ((pos[t] * turns[i]) % (1 << 64)) / 2.0 ** 64
            if abs(np.cos(ang)) > 0.8:
                break
        else:
            t, i = 16 * b, 0
            pos[t], ang = 0, 0.0
        d0, d1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        x1 = np.float32(keys[t, 0, d1])
        a = rope.attention_factor
        x0 = np.float32((448.0 * 2.0 ** e + a * float(x1) * np.sin(ang)) / (a * np.cos(ang)))
        for _ in range(b % 5):
            x0 = np.nextafter(x0, np.float32((-1) ** (b // 5) * np.inf))
        keys[t, 0, d0], keys[t, 0, d1] = x0, x1
        y = a * (float(x0) * np.cos(ang) - float(x1) * np.sin(ang))
        expect[b] = 2.0 ** e if abs(y) <= 448.0 * 2.0 ** e else 2.0 ** (e + 1)
    _check_codes(pkv, rope, pos, torch.from_numpy(keys), interleaved, 0, expect)
