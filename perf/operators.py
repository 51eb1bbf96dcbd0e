"""Measured cases of one serving step over an 8-bit paged cache with a scale per block.

Four operators, in the order a step runs them:

  plan     block tables, slots and positions of the step's tokens from the request lengths
  write    rotary positions on the new queries and keys, and the keys' and values' way into the
           pools (float32 or bfloat16 rows, or E4M3 codes with one scale per block and KV head)
  decode   one query token per sequence over an E4M3 pool with block scales
  prefill  a chunk of query tokens per sequence over the same pools, causal

Layouts are the package's: pools [num_blocks][num_kv_heads][16][head_dim], block tables int32
[num_seqs][max_blocks], rows [tokens][heads][head_dim].  A block's scale is the smallest power of
two 2^e, e in [-32, 31], for which its largest magnitude is at most 448 * 2^e.
"""
import math

import torch

own = False

BS = 16
HD = 128          # head_dim of the attention cases
LOG2E = 1.4426950408889634


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a 64-sequence batch: every sequence grows by one token
        dict(name="plan 64 decodes", op="plan", seqs=64, lo=128, hi=2048, chunk=1, chunked=0.0, spare=1.5),
        # a large mixed step: 4096 requests, a tenth of them with prompt chunks of up to 512 tokens
        dict(name="plan 4096 mixed", op="plan", seqs=4096, lo=0, hi=4096, chunk=512, chunked=0.1, spare=1.2),
        # the decode step's rows of the 7B-shaped batch into bfloat16 pools
        dict(name="write 64 rows bf16", op="write", pool="bf16", seqs=64, chunk=1, lo=128, hi=2048, hkv=32, group=1,
             dim=128, rot=128, interleaved=False, scaling="none", base=10000.0, factor=1.0),
        # 70B-shaped decode rows into block-scaled E4M3 pools: part-filled blocks grow by a row
        dict(name="write 256 rows e4m3", op="write", pool="e4m3", seqs=256, chunk=1, lo=512, hi=4096, hkv=8, group=8,
             dim=128, rot=128, interleaved=False, scaling="by_parts", base=10000.0, factor=8.0),
        # the prompt chunks of the 70B-shaped mix, far positions, block-scaled E4M3 pools
        dict(name="write 16x512 rows e4m3", op="write", pool="e4m3", seqs=16, chunk=512, lo=0, hi=131072, hkv=8, group=8,
             dim=128, rot=128, interleaved=False, scaling="by_parts", base=500000.0, factor=8.0),
        # an odd ragged step in float32: interleaved pairs, half of the head rotated
        dict(name="write 7x111 rows f32", op="write", pool="f32", seqs=7, chunk=111, lo=0, hi=1000, hkv=4, group=3,
             dim=64, rot=32, interleaved=True, scaling="linear", base=10000.0, factor=2.0),
        # one short request: latency
        dict(name="decode 1 sequence", op="decode", seqs=1, lo=777, hi=777, hkv=8, group=4, window=0),
        # the 7B-shaped batch
        dict(name="decode 64 MHA", op="decode", seqs=64, lo=128, hi=2048, hkv=32, group=1, window=0),
        # the 70B-shaped batch
        dict(name="decode 256 GQA", op="decode", seqs=256, lo=512, hi=4096, hkv=8, group=8, window=0),
        # few long contexts
        dict(name="decode 8 long", op="decode", seqs=8, lo=32768, hi=32768, hkv=32, group=1, window=0),
        # ragged small chunks on short contexts: latency
        dict(name="prefill 3 ragged", op="prefill", seqs=3, chunk=130, even=False, lo=0, hi=400, hkv=8, group=4, window=0),
        # the 70B-shaped chunked mix
        dict(name="prefill 16x512 GQA", op="prefill", seqs=16, chunk=512, even=True, lo=0, hi=8192, hkv=8, group=8, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "decode", "prefill"])
    if op == "plan":
        seqs = _log(rng, 1, 4096)
        return dict(op=op, seqs=seqs, lo=0, hi=_log(rng, 1, 4096), chunk=_log(rng, 1, 512),
                    chunked=rng.choice([0.0, 0.05, 0.1]), spare=rng.choice([0.7, 1.0, 1.5]))
    if op == "write":
        pool = rng.choice(["f32", "bf16", "e4m3", "e4m3"])
        dim = rng.choice([64, 128, 128, 256])
        hkv, group = rng.choice([1, 2, 4, 8, 32]), rng.choice([1, 2, 3, 4, 8])
        if hkv == 32:
            group = 1
        rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
        seqs = _log(rng, 1, 256)
        rows = 16 * 512 * 80 * 128 // (hkv * (group + 2) * dim * (2 if pool == "f32" else 1))
        chunk = _log(rng, 1, max(2, min(2048, rows // seqs)))
        scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
        return dict(op=op, pool=pool, seqs=seqs, chunk=chunk, lo=0, hi=_log(rng, 16, 131072), hkv=hkv, group=group,
                    dim=dim, rot=rot, interleaved=rng.random() < 0.5, scaling=scaling,
                    base=rng.choice([10000.0, 500000.0]), factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0]))
    if op == "decode":
        hkv, group = rng.choice([(1, 8), (2, 7), (4, 5), (4, 2), (8, 8), (8, 4), (8, 3), (8, 6), (16, 1), (32, 1)])
        seqs = _log(rng, 1, 256)
        hi = _log(rng, 1, max(2, min(32768, 256 * 2304 * 8 // (seqs * hkv))))
        return dict(op=op, seqs=seqs, lo=rng.choice([0, 1, hi // 2]), hi=hi, hkv=hkv, group=group,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
    hkv, group = rng.choice([(1, 16), (2, 8), (4, 2), (8, 8), (8, 4), (8, 1), (16, 2), (32, 1)])
    seqs = _log(rng, 1, 16)
    chunk = _log(rng, 1, 2048)
    hi = rng.randint(0, 8192)
    while seqs * chunk * hkv * group * (hi + chunk) > 16 * 512 * 64 * 8192:
        chunk, hi = max(1, chunk // 2), hi * 3 // 4
    return dict(op=op, seqs=seqs, chunk=chunk, even=rng.random() < 0.5, lo=0, hi=hi, hkv=hkv, group=group,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _host(case, seed):
    return torch.Generator().manual_seed(seed * 7919 + 13)


def _lengths(case):
    """Every sequence's tokens before the step and in it (int64, host): the case's own, so that
    shapes and work are the same for every seed; prepare() deals them out in the seed's order."""
    g, n, op, chunk = torch.Generator().manual_seed(4711), case["seqs"], case["op"], case.get("chunk", 1)
    ints = lambda lo, hi: torch.randint(int(lo), int(hi) + 1, (n,), generator=g)  # noqa: E731
    lens = ints(case["lo"], case["hi"])
    if op == "plan":
        return lens, torch.where(torch.rand(n, generator=g) < case["chunked"], ints(0, chunk), torch.ones(n, dtype=torch.int64))
    if op == "write" and chunk % 2:
        return lens, ints(max(1, chunk // 2), chunk)
    if op == "prefill" and not case["even"]:
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
    """E4M3 codes and block scales of normal values whose size varies from block to block."""
    codes = torch.empty(blocks, hkv, BS, dim, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(blocks, hkv, device="cuda")
    step = max(1, (1 << 27) // (hkv * BS * dim))
    for a in range(0, blocks, step):
        b = min(blocks, a + step)
        x = torch.randn(b - a, hkv, BS, dim, device="cuda", generator=gpu)
        x *= torch.exp2(0.7 * torch.randn(b - a, hkv, 1, 1, device="cuda", generator=gpu))
        s = _block_scale(x.abs().amax((2, 3)))
        codes[a:b] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
        scales[a:b] = s
    return codes, scales


def _block_scale(amax):
    """Smallest 2^e, e in [-32, 31], with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax / 448)      # amax / 448 = m * 2^e, m in [0.5, 1): 2^e bounds it, 2^(e-1) only at m = 0.5
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, -32)).clamp(-32, 31)
    return torch.ldexp(torch.ones_like(amax), e)


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
    g = _host(case, seed)
    gpu = torch.Generator("cuda").manual_seed(seed)
    op, n = case["op"], case["seqs"]
    order = torch.randperm(n, generator=g)
    lens, new = (x[order] for x in _lengths(case))
    if op == "plan":
        total, most = int(new.sum()), int((lens + new).max())
        need = int(((lens + new + BS - 1) // BS - (lens + BS - 1) // BS).sum())
        tables, blocks = _tables(g, lens)
        wide = torch.full((n, (most + BS - 1) // BS + 1), -1, dtype=torch.int32)
        wide[:, :min(tables.shape[1], wide.shape[1])] = tables[:, :wide.shape[1]]
        free = torch.randperm(max(1, int(need * case["spare"])), generator=g).to(torch.int32) + blocks
        return dict(op=op, tables=wide.cuda(), lens=lens.to(torch.int32).cuda(), new=new.to(torch.int32).cuda(),
                    free=free.cuda(), num_free=torch.tensor([free.numel()], dtype=torch.int32).cuda(),
                    blocks=blocks + free.numel(), capacity=total + total // 16 + 1)
    hkv, hq = case["hkv"], case["hkv"] * case["group"]
    if op == "write":
        dim, pool = case["dim"], case["pool"]
        first = lens // BS                       # only the blocks that this step touches are in the pool
        need = (lens + new + BS - 1) // BS - first
        blocks = int(need.sum() + n // 8 + 1)
        perm = torch.randperm(blocks, generator=g)
        seq = torch.repeat_interleave(torch.arange(n), new)
        row = torch.arange(int(new.sum())) - (new.cumsum(0) - new)[seq]
        pos = lens[seq] + row
        blk = perm[(need.cumsum(0) - need)[seq] + pos // BS - first[seq]]
        slots = blk * BS + pos % BS
        dt = torch.float32 if pool == "f32" else torch.bfloat16
        t = int(new.sum())
        # the projections' output holds q, k and v of a token side by side
        qkv = torch.randn(t, hq + 2 * hkv, dim, device="cuda", generator=gpu)
        qkv *= torch.exp2(0.7 * torch.randn(t, hq + 2 * hkv, 1, device="cuda", generator=gpu))
        qkv = qkv.to(dt)
        s = dict(op=op, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], pos=pos.to(torch.int32).cuda(),
                 slots=slots.cuda(), interleaved=case["interleaved"], runs=int(need.sum()))
        if pool == "e4m3":
            s["kc"], s["ks"] = _pool(gpu, blocks, hkv, dim)
            s["vc"], s["vs"] = _pool(gpu, blocks, hkv, dim)
        else:
            s["kc"] = torch.randn(blocks, hkv, BS, dim, device="cuda", generator=gpu).to(dt)
            s["vc"] = torch.randn(blocks, hkv, BS, dim, device="cuda", generator=gpu).to(dt)
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
    s = dict(op=op, tables=tables.cuda(), lens=lens.to(torch.int32).cuda(), window=case["window"], scale=HD ** -0.5)
    s["kc"], s["ks"] = _pool(gpu, blocks, hkv, HD)
    s["vc"], s["vs"] = _pool(gpu, blocks, hkv, HD)
    rows = n
    if op == "prefill":
        start = torch.zeros(n + 1, dtype=torch.int64)
        start[1:] = new.cumsum(0)
        rows = int(start[-1])
        s["start"], s["longest"] = start.to(torch.int32).cuda(), int(new.max())
    s["q"] = torch.randn(rows, hq, HD, device="cuda", generator=gpu).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        import paged_kv_cache_100_gb300 as pkv
        if s["op"] == "plan":
            p = pkv.plan_step(s["tables"], s["lens"], s["new"], s["free"], s["num_free"], s["capacity"], s["blocks"])
            return dict(tables=s["tables"], lens=p.context_lens, start=p.query_start, slots=p.slot_mapping,
                        pos=p.positions, free=p.num_free)
        if s["op"] == "write":
            q = pkv.rope_cache_write(s["q"], s["k"], s["v"], s["pos"], s["rope"], s["kc"], s["vc"], s["slots"],
                                     k_scales=s.get("ks"), v_scales=s.get("vs"))
            return {k: v for k, v in dict(q=q, kc=s["kc"], vc=s["vc"], ks=s.get("ks"), vs=s.get("vs")).items() if v is not None}
        if s["op"] == "decode":
            return pkv.decode_block_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["tables"], s["lens"], s["scale"],
                                        window=s["window"])
        return pkv.prefill_block_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["tables"], s["lens"], s["start"],
                                     s["longest"], s["scale"], window=s["window"])
    return {"plan": _plan, "write": _write, "decode": _decode, "prefill": _prefill}[s["op"]](s)


def _plan(s):
    tables, lens, new = s["tables"], s["lens"].long(), s["new"].long()
    n, width = tables.shape
    have = (lens + BS - 1) // BS
    need = (lens + new + BS - 1) // BS - have
    blocks, tokens = need.cumsum(0), new.cumsum(0)
    free = s["num_free"].long()
    served = (blocks <= free) & (tokens <= s["capacity"])
    new = new * served
    start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    col = torch.arange(width, device=tables.device)[None, :] - have[:, None]
    fresh = (col >= 0) & (col < (need * served)[:, None])
    at = (free - 1 - (blocks - need)[:, None] - col).clamp(0, s["free"].numel() - 1)
    tables.copy_(torch.where(fresh, s["free"][at], tables))
    i = torch.arange(s["capacity"], device=tables.device)
    seq = torch.searchsorted(start[1:], i, right=True)
    real = seq < n
    seq = seq.clamp(max=n - 1)
    pos = torch.where(real, lens[seq] + i - start[seq], torch.zeros_like(i))
    slots = tables[seq, pos // BS].long() * BS + pos % BS
    return dict(tables=tables, lens=(lens + new).int(), start=start.int(), slots=torch.where(real, slots, -torch.ones_like(slots)),
                pos=pos.int(), free=(free - (need * served).sum()).int())


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
    if "ks" not in s:
        k = _turned(s["k"].float(), cos.float(), sin.float(), s["interleaved"])
        s["kc"][blk, :, off] = k.to(s["kc"].dtype)
        s["vc"][blk, :, off] = s["v"]
        return dict(q=q, kc=s["kc"], vc=s["vc"])
    k = _turned(s["k"].double(), cos, sin, s["interleaved"])   # next to a code's border: in 64 bits
    first = torch.ones_like(blk, dtype=torch.bool)
    first[1:] = blk[1:] != blk[:-1]
    run_of = first.cumsum(0) - 1
    low = torch.full((s["runs"],), BS, device=blk.device).scatter_reduce(0, run_of, off, "amin")
    ids = torch.zeros_like(low).scatter(0, run_of, blk)
    for rows, pool, scales in ((k, s["kc"], s["ks"]), (s["v"].double(), s["vc"], s["vs"])):
        fresh = torch.zeros((s["runs"], rows.shape[1], BS, rows.shape[2]), dtype=rows.dtype, device=rows.device)
        fresh[run_of, :, off] = rows
        old = scales[ids]
        scale = _block_scale(fresh.abs().amax((2, 3)).float())
        scale = torch.where(low[:, None] > 0, torch.maximum(old, scale), scale)
        codes = pool.view(torch.uint8)[ids]
        kept = codes.view(torch.float8_e4m3fn).double() * (old / scale)[:, :, None, None]
        put = torch.zeros((s["runs"], BS), dtype=torch.bool, device=rows.device)
        put[run_of, off] = True
        value = torch.where(put[:, None, :, None], fresh / scale[:, :, None, None], kept)
        change = put | (torch.arange(BS, device=rows.device) < low[:, None])
        coded = value.float().to(torch.float8_e4m3fn).view(torch.uint8)
        pool.view(torch.uint8)[ids] = torch.where(change[:, None, :, None], coded, codes)
        scales[ids] = scale
    return dict(q=q, kc=s["kc"], vc=s["vc"], ks=s["ks"], vs=s["vs"])


def _gathered(codes, scales, tables):
    """Rows of every table in order, float32 [seqs][heads][positions][dim]."""
    at = tables.long().clamp(min=0)
    x = codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    x *= scales[at][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _softmax(score, seen):
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    w = torch.exp(score - top)
    return w / w.sum(-1, keepdim=True).clamp(min=1e-30)


def _decode(s):
    n, hq, d = s["q"].shape
    k, v = _gathered(s["kc"], s["ks"], s["tables"]), _gathered(s["vc"], s["vs"], s["tables"])
    hkv = k.shape[1]
    score = s["q"].float().view(n, hkv, hq // hkv, d) @ k.transpose(-1, -2) * s["scale"]
    pos, lens = torch.arange(k.shape[2], device=k.device), s["lens"].long()[:, None, None, None]
    seen = (pos < lens) & (pos >= lens - s["window"] if s["window"] else pos >= 0)
    v = v.masked_fill(~seen.transpose(-1, -2), 0)
    return (_softmax(score, seen) @ v).reshape(n, hq, d).to(s["q"].dtype)


def _prefill(s):
    rows, hq, d = s["q"].shape
    k, v = _gathered(s["kc"], s["ks"], s["tables"]), _gathered(s["vc"], s["vs"], s["tables"])
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
    v = v.masked_fill(pos[:, None] >= lens[:, None, None, None], 0)
    o = _softmax(q @ k.transpose(-1, -2) * s["scale"], seen) @ v
    o = o.view(n, hkv, s["longest"], hq // hkv, d).transpose(1, 2).flatten(2, 3)
    return o[seq, row].to(s["q"].dtype)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    op, n = case["op"], case["seqs"]
    lens, new = _lengths(case)
    grown = float(((lens + new + BS - 1) // BS - (lens + BS - 1) // BS).sum())
    part = float(((lens % BS) * (new > 0)).sum())             # rows of part-filled last blocks
    lens, new = lens.double(), new.double()
    t = float(new.sum())
    if op == "plan":                                          # lengths in and out, free blocks into tables, slots, positions
        return {"bytes": n * 16 + grown * 8 + t * 12, "flops": 0}
    hkv, hq = case["hkv"], case["hkv"] * case["group"]
    if op == "write":
        size, out = (4, 4) if case["pool"] == "f32" else (2, 2) if case["pool"] == "bf16" else (2, 1)
        bytes_ = t * case["dim"] * (2 * hq * size + 2 * hkv * (size + out)) + t * 12
        if case["pool"] == "e4m3":                            # scales; earlier rows are read where their block's scale grows
            bytes_ += n * hkv * 16 + 0.25 * part * 2 * hkv * case["dim"] * 2
        return {"bytes": bytes_, "flops": t * (hq + hkv) * case["rot"] * 3}
    scale = 2 * 4 / (BS * HD)
    if op == "decode":
        seen = float((lens.clamp(max=case["window"]) if case["window"] else lens).sum())
        return {"bytes": seen * hkv * HD * (2 + scale) + n * hq * HD * 4 + seen / BS * 4, "flops": 4 * HD * hq * seen}
    seen, read = lens + (new + 1) / 2, lens + new
    if case["window"]:
        seen, read = seen.clamp(max=case["window"]), torch.minimum(read, case["window"] + new)
    return {"bytes": float(read.sum()) * hkv * HD * (2 + scale) + t * hq * HD * 4,
            "flops": 4 * HD * hq * float((new * seen).sum())}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "write":
        return _exact_write(case, s)
    k, v = s["kc"].view(torch.uint8), s["vc"].view(torch.uint8)
    q, out = s["q"].double(), torch.zeros_like(s["q"], dtype=torch.float64)
    group = case["group"]
    for b, length in enumerate(s["lens"].tolist()):
        at = s["tables"][b, :(length + BS - 1) // BS].long()
        rows = slice(b, b + 1) if case["op"] == "decode" else slice(*s["start"][b:b + 2].tolist())
        if length == 0 or rows.start == rows.stop:
            continue
        last = torch.arange(length - (rows.stop - rows.start), length, device="cuda")[:, None]
        pos = torch.arange(length, device="cuda")[None, :]
        hidden = pos > last
        if case["window"]:
            hidden |= pos + case["window"] <= last
        for h in range(case["hkv"]):
            kh = (k[at, h].view(torch.float8_e4m3fn).double() * s["ks"][at, h].double()[:, None, None]).flatten(0, 1)[:length]
            vh = (v[at, h].view(torch.float8_e4m3fn).double() * s["vs"][at, h].double()[:, None, None]).flatten(0, 1)[:length]
            for j in range(h * group, (h + 1) * group):
                p = torch.softmax((q[rows, j] @ kh.T * s["scale"]).masked_fill(hidden, -math.inf), -1)
                out[rows, j] = p @ vh
    return out


def _exact_write(case, s):
    inv, a = _frequencies(case)
    turn = torch.polar(torch.full((), float(a), dtype=torch.float64), torch.outer(s["pos"].cpu().double(), inv)).cuda()[:, None]
    half = case["rot"] // 2

    def turned(x):
        y = x.double().clone()
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :case["rot"]].unflatten(-1, (half, 2)).contiguous()) * turn
            y[..., :case["rot"]] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * turn
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    out = dict(q=turned(s["q"]), kc=s["kc"].double(), vc=s["vc"].double())
    k, v, slots = turned(s["k"]), s["v"].double(), s["slots"].tolist()
    if case["pool"] != "e4m3":
        blk, off = torch.tensor(slots).cuda() // BS, torch.tensor(slots).cuda() % BS
        out["kc"][blk, :, off], out["vc"][blk, :, off] = k, v
        return out
    ends = [i for i in range(len(slots)) if i + 1 == len(slots) or slots[i + 1] // BS != slots[i] // BS]
    new = {}
    for name, x in (("k", k), ("v", v)):
        pool, scales = out[name + "c"], s[name + "s"].double()
        top = x.abs().amax(-1)
        a = 0
        amax = torch.stack([top[i:j + 1].amax(0) for i, j in zip([0] + [e + 1 for e in ends[:-1]], ends)]).cpu()
        e = torch.ceil(torch.log2((amax / 448).clamp(min=2.0 ** -32))).clamp(-32, 31)
        e = torch.where(amax <= 448 * torch.exp2(e - 1), (e - 1).clamp(min=-32), e)
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e).clamp(-32, 31)
        want = torch.exp2(e).cuda()
        for r, end in enumerate(ends):
            block, low, count = slots[a] // BS, slots[a] % BS, end + 1 - a
            scale = torch.maximum(want[r], scales[block]) if low else want[r]
            pool[block, :, :low] *= (scales[block] / scale)[:, None, None]
            pool[block, :, low:low + count] = x[a:end + 1].transpose(0, 1) / scale[:, None, None]
            pool[block, :, :low + count] = pool[block, :, :low + count].float().to(torch.float8_e4m3fn).double()
            scales[block] = scale
            a = end + 1
        new[name + "s"] = scales
    return dict(out, **new)
