"""Measured cases of a serving step over a paged KV cache held in 4 bits.

Four operators:

  write    rotary positions on the new queries and keys, and the keys' and values' way into the pools;
           the pools' values are read back in the same pass, as its output
  read     the blocks of every sequence's context as bfloat16 or float32 rows, in blocks of their own
  decode   one query token per sequence over the 4-bit pools
  prefill  a chunk of query tokens per sequence over the same pools, causal

A pool is uint8 [num_blocks][num_kv_heads][16][9 * head_dim / 16]: the 9 * head_dim bytes of a block's
tile of one KV head are the codes of its 16 rows (two E2M1 codes a byte, the even element in the low
half), then its 16 rows of scales, one byte per 16 elements.  A scale byte is a positive number of 5
exponent and 3 mantissa bits (a float16's bits 14 to 7); an element is its code's value times its scale.
The scale of 16 elements is amax / 6 rounded to nearest even, at least 2^-17 (0 where amax is 0), at
most 10240; a code is the nearest one to element / scale, ties to even, 6 at most.
"""
import math

import torch

own = False

BS = 16
CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step's rows of the 7B-shaped batch: latency
        dict(name="write 64 rows", op="write", type="bf16", seqs=64, chunk=1, lo=128, hi=2048, hkv=32, group=1, dim=128,
             rot=128, interleaved=False, scaling="none", base=10000.0, factor=1.0),
        # the prompt chunks of the 70B-shaped mix, far positions
        dict(name="write 16x512 rows", op="write", type="bf16", seqs=16, chunk=512, lo=0, hi=131072, hkv=8, group=8,
             dim=128, rot=128, interleaved=False, scaling="by_parts", base=500000.0, factor=8.0),
        # an odd ragged step in float32: neighbouring pairs, half of the head turned
        dict(name="write 7x111 rows f32", op="write", type="f32", seqs=7, chunk=111, lo=0, hi=1000, hkv=4, group=3,
             dim=64, rot=32, interleaved=True, scaling="linear", base=10000.0, factor=2.0),
        # one short context read back: latency
        dict(name="read 1 context f32", op="read", type="f32", seqs=1, lo=777, hi=777, hkv=8, dim=128),
        # the contexts of the 70B-shaped chunked mix
        dict(name="read 16 contexts", op="read", type="bf16", seqs=16, lo=0, hi=8192, hkv=8, dim=128),
        # one short request: latency
        dict(name="decode 1 sequence", op="decode", seqs=1, lo=777, hi=777, hkv=8, group=4, dim=128, window=0),
        # the 7B-shaped batch
        dict(name="decode 64 MHA", op="decode", seqs=64, lo=128, hi=2048, hkv=32, group=1, dim=128, window=0),
        # the 70B-shaped batch
        dict(name="decode 256 GQA", op="decode", seqs=256, lo=512, hi=4096, hkv=8, group=8, dim=128, window=0),
        # small heads, ragged, a window that ends inside blocks
        dict(name="decode 48 window", op="decode", seqs=48, lo=0, hi=5000, hkv=4, group=5, dim=64, window=1111),
        # few long contexts
        dict(name="decode 8 long", op="decode", seqs=8, lo=32768, hi=32768, hkv=32, group=1, dim=128, window=0),
        # ragged small chunks on short contexts: latency
        dict(name="prefill 3 ragged", op="prefill", seqs=3, chunk=130, even=False, lo=0, hi=400, hkv=8, group=4, dim=128,
             window=0),
        # the 70B-shaped chunked mix
        dict(name="prefill 16x512 GQA", op="prefill", seqs=16, chunk=512, even=True, lo=0, hi=8192, hkv=8, group=8, dim=128,
             window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "prefill"])
    if op == "write":
        kind = rng.choice(["f32", "bf16", "bf16"])
        dim = rng.choice([64, 128, 128, 256])
        hkv, group = rng.choice([1, 2, 4, 8, 32]), rng.choice([1, 2, 3, 4, 8])
        if hkv == 32:
            group = 1
        rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
        seqs = _log(rng, 1, 256)
        rows = 16 * 512 * 80 * 128 // (hkv * (group + 2) * dim * (2 if kind == "f32" else 1))
        chunk = _log(rng, 1, max(2, min(2048, rows // seqs)))
        scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
        return dict(op=op, type=kind, seqs=seqs, chunk=chunk, lo=0, hi=_log(rng, 16, 131072), hkv=hkv, group=group,
                    dim=dim, rot=rot, interleaved=rng.random() < 0.5, scaling=scaling,
                    base=rng.choice([10000.0, 500000.0]), factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0]))
    if op == "read":
        hkv, dim, seqs = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128, 128, 256]), _log(rng, 1, 64)
        return dict(op=op, type=rng.choice(["f32", "bf16", "bf16"]), seqs=seqs, lo=rng.choice([0, 1]), hkv=hkv, dim=dim,
                    hi=_log(rng, 1, max(2, min(32768, 16 * 4096 * 8 * 128 // (seqs * hkv * dim)))))
    if op == "decode":
        hkv, group = rng.choice([(1, 8), (2, 7), (4, 5), (4, 2), (8, 8), (8, 4), (8, 3), (8, 6), (16, 1), (32, 1), (2, 16)])
        dim, seqs = rng.choice([64, 128, 128, 128, 256]), _log(rng, 1, 256)
        hi = _log(rng, 1, max(2, min(32768, 256 * 2304 * 8 * 128 // (seqs * hkv * dim))))
        return dict(op=op, seqs=seqs, lo=rng.choice([0, 1, hi // 2]), hi=hi, hkv=hkv, group=group, dim=dim,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
    hkv, group = rng.choice([(1, 16), (2, 8), (4, 2), (8, 8), (8, 4), (8, 1), (16, 2), (32, 1)])
    seqs = _log(rng, 1, 16)
    chunk = _log(rng, 1, 2048)
    hi = rng.randint(0, 8192)
    while seqs * chunk * hkv * group * (hi + chunk) > 16 * 512 * 64 * 8192:
        chunk, hi = max(1, chunk // 2), hi * 3 // 4
    return dict(op=op, seqs=seqs, chunk=chunk, even=rng.random() < 0.5, lo=0, hi=hi, hkv=hkv, group=group, dim=128,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _lengths(case):
    """Every sequence's tokens before the step and in it (int64, host): the case's own, so that
    shapes and work are the same for every seed; prepare() deals them out in the seed's order."""
    g, n, chunk = torch.Generator().manual_seed(4711), case["seqs"], case.get("chunk", 1)
    ints = lambda lo, hi: torch.randint(int(lo), int(hi) + 1, (n,), generator=g)  # noqa: E731
    lens = ints(case["lo"], case["hi"])
    if case["op"] == "write" and chunk % 2:
        return lens, ints(max(1, chunk // 2), chunk)
    if case["op"] == "prefill" and not case["even"]:
        return lens, ints(1, chunk)
    return lens, torch.full((n,), chunk)


def _tables(g, lens, spare=0.1):
    """Block tables of `lens` tokens (int64, host): slices of a shuffled pool, -1 behind."""
    need = (lens + BS - 1) // BS
    width = max(1, int(need.max()))
    blocks = max(1, int(need.sum() * (1 + spare)) + 1)
    perm = torch.randperm(blocks, generator=g)
    start = need.cumsum(0) - need
    col = torch.arange(width)[None, :]
    at = (start[:, None] + col).clamp(max=blocks - 1)
    return torch.where(col < need[:, None], perm[at], torch.full_like(at, -1)).to(torch.int32), blocks


def _pool(gpu, blocks, hkv, dim):
    """A pool of normal values whose size varies from row to row."""
    pool = torch.empty(blocks, hkv, 9 * dim, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (hkv * BS * dim))
    for a in range(0, blocks, step):
        b = min(blocks, a + step)
        x = torch.randn(b - a, hkv, BS, dim, device="cuda", generator=gpu)
        x *= torch.exp2(0.7 * torch.randn(b - a, hkv, BS, 1, device="cuda", generator=gpu))
        codes, scales = _encoded(x)
        pool[a:b, :, :8 * dim], pool[a:b, :, 8 * dim:] = codes.flatten(2), scales.flatten(2)
    return pool.view(blocks, hkv, BS, 9 * dim // 16)


def _frequencies(case):
    """Rotary angles per position (radians, float64) and the factor on cos and sin."""
    d, base, f = case["rot"], case["base"], case["factor"]
    i = torch.arange(d // 2, dtype=torch.float64)
    if case["scaling"] == "ntk" and d > 2:
        base = base * f ** (d / (d - 2))
    inv = base ** (-2.0 * i / d)
    if case["scaling"] == "linear":
        return inv / f, 1.0
    if case["scaling"] == "by_parts":
        at = lambda turns: d * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), d - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return inv * (1 - ramp) + inv / f * ramp, 0.1 * math.log(f) + 1.0
    return inv, 1.0


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    gpu = torch.Generator("cuda").manual_seed(seed)
    op, n, hkv, dim = case["op"], case["seqs"], case["hkv"], case["dim"]
    order = torch.randperm(n, generator=g)
    lens, new = (x[order] for x in _lengths(case))
    if op == "write":
        hq = hkv * case["group"]
        first = lens // BS                       # only the blocks that this step touches are in the pool
        need = (lens + new + BS - 1) // BS - first
        blocks = int(need.sum() + n // 8 + 1)
        perm = torch.randperm(blocks, generator=g)
        seq = torch.repeat_interleave(torch.arange(n), new)
        pos = lens[seq] + torch.arange(int(new.sum())) - (new.cumsum(0) - new)[seq]
        slots = perm[(need.cumsum(0) - need)[seq] + pos // BS - first[seq]] * BS + pos % BS
        dt, t = torch.float32 if case["type"] == "f32" else torch.bfloat16, int(new.sum())
        # the projections' output holds q, k and v of a token side by side
        qkv = torch.randn(t, hq + 2 * hkv, dim, device="cuda", generator=gpu)
        qkv *= torch.exp2(0.7 * torch.randn(t, hq + 2 * hkv, 1, device="cuda", generator=gpu))
        qkv = qkv.to(dt)
        s = dict(op=op, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], pos=pos.to(torch.int32).cuda(),
                 slots=slots.cuda(), interleaved=case["interleaved"], kc=_pool(gpu, blocks, hkv, dim),
                 vc=_pool(gpu, blocks, hkv, dim), tables=torch.arange(blocks, dtype=torch.int32, device="cuda")[None],
                 lens=torch.tensor([blocks * BS], dtype=torch.int32, device="cuda"))
        if own:
            import paged_kv_cache_100_gb300 as pkv
            s["rope"] = pkv.rotary_plan(case["rot"], case["base"], interleaved=case["interleaved"],
                                        scaling=case["scaling"], factor=case["factor"], original_context=4096,
                                        device="cuda")
        else:
            inv, a = _frequencies(case)
            s["inv"], s["a"] = inv.cuda(), a
        return s
    if op == "prefill":
        lens = lens + new
    tables, blocks = _tables(g, lens)
    s = dict(op=op, tables=tables.cuda(), lens=lens.to(torch.int32).cuda(), kc=_pool(gpu, blocks, hkv, dim),
             vc=_pool(gpu, blocks, hkv, dim))
    if op == "read":                             # blocks of a prefill's own, kept from step to step
        shape = (n * tables.shape[1], hkv, BS, dim)
        dt = torch.float32 if case["type"] == "f32" else torch.bfloat16
        s["ko"], s["vo"] = torch.zeros(shape, dtype=dt, device="cuda"), torch.zeros(shape, dtype=dt, device="cuda")
        return s
    s["window"], s["scale"] = case["window"], dim ** -0.5
    rows = n
    if op == "prefill":
        start = torch.zeros(n + 1, dtype=torch.int64)
        start[1:] = new.cumsum(0)
        rows = int(start[-1])
        s["start"], s["longest"] = start.to(torch.int32).cuda(), int(new.max())
    s["q"] = torch.randn(rows, hkv * case["group"], dim, device="cuda", generator=gpu).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        import paged_kv_cache_100_gb300 as pkv
        if s["op"] == "write":
            q = pkv.rope_cache_write_fp4(s["q"], s["k"], s["v"], s["pos"], s["rope"], s["kc"], s["vc"], s["slots"])
            k, v = pkv.cache_read_fp4(s["kc"], s["vc"], s["tables"], s["lens"], dtype=torch.bfloat16)
            return dict(q=q, k=k, v=v)
        if s["op"] == "read":
            k, v = pkv.cache_read_fp4(s["kc"], s["vc"], s["tables"], s["lens"], key_out=s["ko"], value_out=s["vo"])
            return dict(k=k, v=v)
        if s["op"] == "decode":
            return pkv.decode_fp4(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["scale"], window=s["window"])
        return pkv.prefill_fp4(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["start"], s["longest"], s["scale"],
                               window=s["window"])
    return {"write": _write, "read": _read, "decode": _decode, "prefill": _prefill}[s["op"]](s)


def _encoded(x):
    """Code bytes [..., dim / 2] and scale bytes [..., dim / 16] of rows [..., dim]."""
    group = x.unflatten(-1, (-1, 16))
    amax = group.abs().amax(-1)
    q = amax / 6
    step = torch.exp2((torch.frexp(q)[1] - 1).clamp(min=-14).to(q.dtype) - 3)
    scale = (torch.round(q / step) * step).clamp(min=2.0 ** -17, max=10240.0)
    scale = torch.where(amax > 0, scale, torch.zeros_like(scale))
    y = torch.where(amax[..., None] > 0, group / scale[..., None], torch.zeros_like(group))
    mag = y.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0)).to(y.dtype)
    mag = (torch.round(mag / step) * step).clamp(max=6.0)
    code = torch.bucketize(mag.float(), torch.tensor(CODES, device=x.device)) + 8 * (y < 0)
    code = code.flatten(-2).unflatten(-1, (-1, 2)).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), (scale.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)


def _decoded(pool, at=None):
    """Values (float32) of the pool's tiles, or of blocks `at`: [...][num_kv_heads][16][head_dim]."""
    tile = pool.flatten(2) if at is None else pool.flatten(2)[at]
    dim = tile.shape[-1] // 9
    scale = (tile[..., 8 * dim:].to(torch.int16) << 7).view(torch.float16).float()
    byte = torch.arange(256, device=pool.device)
    value = torch.tensor(CODES + [-c for c in CODES], device=pool.device)
    pairs = torch.stack([value[byte & 15], value[byte >> 4]], -1)
    x = pairs[tile[..., :8 * dim].int()].flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2).unflatten(-1, (BS, dim))


def _turned(x, cos, sin, interleaved):
    half = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _write(s):
    angle = s["pos"].double()[:, None, None] * s["inv"]        # far positions: the angle in 64 bits
    cos, sin = torch.cos(angle) * s["a"], torch.sin(angle) * s["a"]
    q = _turned(s["q"].float(), cos.float(), sin.float(), s["interleaved"]).to(s["q"].dtype)
    blk, off = s["slots"] // BS, s["slots"] % BS
    k = _turned(s["k"].double(), cos, sin, s["interleaved"])   # next to a code's border: in 64 bits
    for rows, pool in ((k, s["kc"]), (s["v"].double(), s["vc"])):
        codes, scales = _encoded(rows)
        tiles, dim = pool.flatten(2), rows.shape[-1]
        tiles[..., :8 * dim].unflatten(-1, (BS, -1))[blk, :, off] = codes
        tiles[..., 8 * dim:].unflatten(-1, (BS, -1))[blk, :, off] = scales
    return dict(q=q, k=_decoded(s["kc"]).to(torch.bfloat16), v=_decoded(s["vc"]).to(torch.bfloat16))


def _read(s):
    n, width = s["tables"].shape
    lens = s["lens"].long()[:, None]
    entry = torch.arange(width, device=lens.device)[None, :]
    held = entry * BS < lens
    row = entry[..., None] * BS + torch.arange(BS, device=lens.device) < lens[..., None]
    at = s["tables"].long()[held]
    for pool, out in ((s["kc"], s["ko"]), (s["vc"], s["vo"])):
        x = torch.where(row[held][:, None, :, None], _decoded(pool, at), 0.0)     # behind the context: zeros
        out.unflatten(0, (n, width))[held] = x.to(out.dtype)
    return dict(k=s["ko"], v=s["vo"])


def _gathered(pool, tables):
    """Rows of every table in order, float32 [seqs][heads][positions][dim]."""
    return _decoded(pool, tables.long().clamp(min=0)).permute(0, 2, 1, 3, 4).flatten(2, 3)


def _softmax(score, seen):
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    w = torch.exp(score - top)
    return w / w.sum(-1, keepdim=True).clamp(min=1e-30)


def _decode(s):
    n, hq, d = s["q"].shape
    k, v = _gathered(s["kc"], s["tables"]), _gathered(s["vc"], s["tables"])
    hkv = k.shape[1]
    score = s["q"].float().view(n, hkv, hq // hkv, d) @ k.transpose(-1, -2) * s["scale"]
    pos, lens = torch.arange(k.shape[2], device=k.device), s["lens"].long()[:, None, None, None]
    seen = (pos < lens) & (pos >= lens - s["window"] if s["window"] else pos >= 0)
    return (_softmax(score, seen) @ v).reshape(n, hq, d).to(s["q"].dtype)


def _prefill(s):
    rows, hq, d = s["q"].shape
    k, v = _gathered(s["kc"], s["tables"]), _gathered(s["vc"], s["tables"])
    n, hkv = k.shape[:2]
    start, lens = s["start"].long(), s["lens"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(rows, device=k.device)
    seq = torch.searchsorted(start[1:], i, right=True)
    row = i - start[seq]
    q = torch.zeros(n, s["longest"], hq, d, device=k.device)
    q[seq, row] = s["q"].float()
    q = q.view(n, -1, hkv, hq // hkv, d).transpose(1, 2).flatten(2, 3)          # [seq][kv head][row, head][dim]
    at = (lens - new)[:, None] + torch.arange(s["longest"], device=k.device)
    pos, at = torch.arange(k.shape[2], device=k.device), at.repeat_interleave(hq // hkv, 1)[:, None, :, None]
    seen = (pos <= at) & (pos < lens[:, None, None, None])
    if s["window"]:
        seen &= pos > at - s["window"]
    o = _softmax(q @ k.transpose(-1, -2) * s["scale"], seen) @ v
    o = o.view(n, hkv, s["longest"], hq // hkv, d).transpose(1, 2).flatten(2, 3)
    return o[seq, row].to(s["q"].dtype)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    op, n, hkv, dim = case["op"], case["seqs"], case["hkv"], case["dim"]
    lens, new = _lengths(case)
    row = 2 * hkv * dim * 9 / 16                              # bytes of a token's keys and values in the pools
    if op == "write":                                         # the rows in, the queries out, the pools' values out
        blocks = int(((lens + new + BS - 1) // BS - lens // BS).sum() + n // 8 + 1)
        size, hq, t = 4 if case["type"] == "f32" else 2, hkv * case["group"], float(new.sum())
        held = blocks * BS
        return {"bytes": t * dim * size * (2 * hq + 2 * hkv) + t * (row + 12) + held * (row + 2 * hkv * dim * 2),
                "flops": t * (hq + hkv) * case["rot"] * 3}
    lens, new = lens.double(), new.double()
    if op == "read":
        held = float(((lens / BS).ceil() * BS).sum())
        return {"bytes": float(lens.sum()) * row + held * 2 * hkv * dim * (4 if case["type"] == "f32" else 2), "flops": 0}
    hq = hkv * case["group"]
    if op == "decode":
        seen = float((lens.clamp(max=case["window"]) if case["window"] else lens).sum())
        return {"bytes": seen * row + n * hq * dim * 4 + seen / BS * 4, "flops": 4 * dim * hq * seen}
    seen, read = lens + (new + 1) / 2, lens + new
    if case["window"]:
        seen, read = seen.clamp(max=case["window"]), torch.minimum(read, case["window"] + new)
    return {"bytes": float(read.sum()) * row + float(new.sum()) * hq * dim * 4,
            "flops": 4 * dim * hq * float((new * seen).sum())}


def _rows64(tiles, dim):
    """Tiles [blocks][9 dim] of one KV head in 64 bits: [blocks * 16][dim]."""
    byte = tiles[:, :8 * dim].reshape(-1, dim // 2).long()
    nibble = torch.stack([byte % 16, byte // 16], -1).flatten(1)
    e, m = nibble // 2 % 4, nibble % 2
    x = torch.where(e > 0, (1 + 0.5 * m) * 2.0 ** (e.double() - 1), 0.5 * m.double()) * (1 - 2 * (nibble // 8))
    b = tiles[:, 8 * dim:].reshape(-1, dim // 16).long()
    e, m = b // 8, b % 8
    scale = torch.where(e > 0, (8 + m) * 2.0 ** (e.double() - 18), m * 2.0 ** -17)
    return x * scale.repeat_interleave(16, 1)


def exact(case, seed):
    s, dim = prepare(case, seed), case["dim"]
    if case["op"] == "write":
        return _exact_write(case, s)
    lens, tables = s["lens"].tolist(), s["tables"].long()
    k, v = s["kc"].flatten(2), s["vc"].flatten(2)
    if case["op"] == "read":
        out = [torch.zeros(s["ko"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
        for b, length in enumerate(lens):
            used, to = (length + BS - 1) // BS, b * tables.shape[1]
            for h in range(case["hkv"]):
                for pool, o in zip((k, v), out):
                    x = _rows64(pool[tables[b, :used], h], dim)
                    x[length:] = 0
                    o[to:to + used, h] = x.view(used, BS, dim)
        return dict(k=out[0], v=out[1])
    q, out, group = s["q"].double(), torch.zeros_like(s["q"], dtype=torch.float64), case["group"]
    for b, length in enumerate(lens):
        at = tables[b, :(length + BS - 1) // BS]
        rows = slice(b, b + 1) if case["op"] == "decode" else slice(*s["start"][b:b + 2].tolist())
        if length == 0 or rows.start == rows.stop:
            continue
        last = torch.arange(length - (rows.stop - rows.start), length, device="cuda")[:, None]
        pos = torch.arange(length, device="cuda")[None, :]
        hidden = pos > last
        if case["window"]:
            hidden |= pos + case["window"] <= last
        for h in range(case["hkv"]):
            kh, vh = _rows64(k[at, h], dim)[:length], _rows64(v[at, h], dim)[:length]
            for j in range(h * group, (h + 1) * group):
                p = torch.softmax((q[rows, j] @ kh.T * s["scale"]).masked_fill(hidden, -math.inf), -1)
                out[rows, j] = p @ vh
    return out


def _exact_write(case, s):
    inv, a = _frequencies(case)
    turn = torch.polar(torch.full((), float(a), dtype=torch.float64), torch.outer(s["pos"].cpu().double(), inv)).cuda()[:, None]
    half, dim, hkv = case["rot"] // 2, case["dim"], case["hkv"]

    def turned(x):
        y = x.double().clone()
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :case["rot"]].unflatten(-1, (half, 2)).contiguous()) * turn
            y[..., :case["rot"]] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * turn
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    def nearest(x, values):
        """Index of the nearest value (ascending); ties to the even index."""
        up = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
        below, above = x - values[up - 1], values[up] - x
        return torch.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)

    byte = torch.arange(227)                                   # the last one is 10240
    scales = torch.where(byte < 8, byte * 2.0 ** -17, (8 + byte % 8) * 2.0 ** (byte // 8 - 18.0)).double().cuda()
    codes = torch.tensor(CODES, dtype=torch.float64, device="cuda")
    blk, off = s["slots"] // BS, s["slots"] % BS
    out = {"q": turned(s["q"])}
    for name, x, pool in (("k", turned(s["k"]), s["kc"]), ("v", s["v"].double(), s["vc"])):
        g = x.unflatten(-1, (-1, 16))
        top = g.abs().amax(-1)
        at = nearest(top / 6, scales)
        scale = scales[torch.where(top > 0, at.clamp(min=1), 0)][..., None]
        y = torch.sign(g) * codes[nearest(g.abs() / scale.clamp(min=2.0 ** -17), codes)] * scale
        blocks = pool.shape[0]
        held = torch.stack([_rows64(pool.flatten(2)[:, h], dim).view(blocks, BS, dim) for h in range(hkv)], 1)
        held[blk, :, off] = y.flatten(-2)
        out[name] = held
    return out
