"""pa_decode_block_fp8 and pa_prefill_block_fp8: attention over E4M3 pools with one scale per block
and KV head, against 64-bit attention over the same values."""
import numpy as np
import pytest
import torch

from tests import block8_ref as R

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_100_gb300.build import build
    build()
    import paged_kv_cache_100_gb300 as m
    return m


class Pool:
    """Pools, tables and lengths of a batch; codes and scales of slots that hold no token are NaN
    codes and absurd scales."""

    def __init__(self, seed, lens, hkv, spread=1.5, width=None, poison=True):
        g = self.g = torch.Generator().manual_seed(seed)
        self.lens = np.asarray(lens, np.int32)
        self.tables, self.blocks = R.tables_for(g, lens, width=width)
        self.hkv = hkv
        self.kc, self.ks = R.pools(g, self.blocks, hkv, D, spread)
        self.vc, self.vs = R.pools(g, self.blocks, hkv, D, spread)
        if poison:
            live = np.zeros((self.blocks, 16), bool)
            for b, n in enumerate(lens):
                for p in range(int(n)):
                    live[self.tables[b, p // 16], p % 16] = True
            dead = torch.from_numpy(~live)
            self.kc[dead[:, None].expand(-1, hkv, -1)] = 0x7F
            self.vc[dead[:, None].expand(-1, hkv, -1)] = 0xFF
            unused = dead.all(1)
            for s in (self.ks, self.vs):
                s[unused] = float("nan")

    def device(self):
        return [t.cuda() for t in (self.kc, self.vc, self.ks, self.vs)] + [
            torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.lens).cuda()]

    def reference(self, q, rows, scale, window=0, floor=1.0):
        """q [rows][Hq][D] float64; rows: (sequence, last position) of each."""
        group = q.shape[1] // self.hkv
        kv, vv = R.decode_codes(self.kc), R.decode_codes(self.vc)
        ks, vs = self.ks.double().numpy(), self.vs.double().numpy()
        out, bound = np.zeros_like(q), np.zeros_like(q)
        for i, (b, last) in enumerate(rows):
            lo = max(0, last + 1 - window) if window else 0
            for h in range(self.hkv):
                j = slice(h * group, (h + 1) * group)
                out[i, j], bound[i, j] = R.attention(q[i, j], kv[:, h], ks[:, h], vv[:, h], vs[:, h], self.tables[b],
                                                     lo, last + 1, scale, floor)
        return out, bound


def _check(got, ref, bound, what=""):
    err = np.abs(got.double().cpu().numpy() - ref)
    limit = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    assert (err <= limit).all(), (what, float(np.nanmax(err - limit)), np.argwhere(~(err <= limit))[:4].tolist())


def _query(pool, rows, hq):
    return torch.randn(rows, hq, D, generator=pool.g).to(torch.bfloat16)


LENS = [1, 15, 16, 17, 0, 100, 513, 1100, 31]


@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 4), (6, 2), (8, 2), (5, 1), (12, 2), (7, 1), (16, 2), (11, 1), (24, 2), (16, 1)])
@pytest.mark.parametrize("partition", [0, 64, 16384])
def test_decode_matches(pkv, hq, hkv, partition):
    p = Pool(hq * 10 + hkv, LENS, hkv)
    q = _query(p, len(LENS), hq)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.decode_block_fp8(q.cuda(), *p.device(), partition_size=partition, status=status)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(LENS)], D ** -0.5)
    _check(out, ref, bound, f"{hq}/{hkv} P={partition}")
    assert (out[4] == 0).all() and int(status.item()) == 0


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 513, 5000])
@pytest.mark.parametrize("hq,hkv,partition", [(8, 8, 0), (16, 2, 0), (8, 2, 32)])
def test_decode_window(pkv, window, hq, hkv, partition):
    p = Pool(window, LENS, hkv)
    q = _query(p, len(LENS), hq)
    dev = p.device()
    first = [max(0, n - window) // 16 for n in LENS]
    for b, f in enumerate(first):                           # released blocks before the window
        dev[4][b, :f] = -1
    out = pkv.decode_block_fp8(q.cuda(), *dev, window=window, partition_size=partition)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(LENS)], D ** -0.5, window)
    _check(out, ref, bound, f"W={window}")


@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 1)])
def test_decode_scales_of_any_size(pkv, hq, hkv):
    """Value scales over the whole range in one context, an outlier block, scales that are no powers
    of two, tiny and negative key scales."""
    lens = [700, 700, 700, 60]
    p = Pool(3, lens, hkv, poison=False)
    p.vs[:] = torch.exp2(torch.randint(-32, 32, p.vs.shape, generator=p.g).float())
    t = p.tables
    p.vs[t[1, :43]] = torch.rand(43, hkv, generator=p.g) + 0.3
    p.vs[t[1, 20]] = 40000.0
    p.ks[t[1, :43]] = torch.randn(43, hkv, generator=p.g) * 0.01
    p.vs[t[2, :44]] = 2.0 ** -32
    p.vs[t[3, :4]] = 2.0 ** 31
    q = _query(p, len(lens), hq)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.decode_block_fp8(q.cuda(), *p.device(), status=status)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(lens)], D ** -0.5)
    _check(out, ref, bound)
    assert int(status.item()) == 0


@pytest.mark.parametrize("hq,hkv,longest", [(16, 2, 100), (5, 1, 700), (48, 16, 200)])
def test_decode_queries_of_any_size(pkv, hq, hkv, longest):
    """Rows of tiny, mixed and zero queries, with key scales that bring their scores back into the usual range:
    small elements count like any others."""
    lens = [longest, 33, longest // 2, 17, 64, 50, 1] + ([40] * 103 if hq == 48 else [])
    p = Pool(hq + longest, lens, hkv, spread=0.7)
    q = _query(p, len(lens), hq)
    for b, e in enumerate((-17, -26, -60, -96)):             # two of the rows with the first heads as they were
        q[b, b % 2:] = (q[b, b % 2:].float() * 2.0 ** e).to(torch.bfloat16)
        p.ks[p.tables[b, :-(-lens[b] // 16)]] *= 2.0 ** -e
    for b in (1, 3):
        q[b, 0] = 0
    q[4, :, 3] *= 2.0 ** 10                                  # one large element beside the others
    q[5, :, ::2] = (q[5, :, ::2].float() * 2.0 ** -12).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.decode_block_fp8(q.cuda(), *p.device(), status=status)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(lens)], D ** -0.5)
    _check(out, ref, bound)
    assert int(status.item()) == 0


@pytest.mark.parametrize("hq,hkv,partition,longest,seqs", [(8, 2, 0, 400, 7), (14, 2, 64, 400, 7), (16, 1, 0, 3000, 5),
                                                           (32, 16, 0, 200, 60)])
def test_decode_rows_of_a_plan(pkv, hq, hkv, partition, longest, seqs):
    """Rows where query_start puts them: sequences that bring nothing, more than one token, or entries outside the
    rows are passed over, and the rows of no sequence are left alone."""
    from paged_kv_cache_100_gb300 import _lib
    rng = np.random.default_rng(seqs)
    lens = [int(x) for x in rng.integers(1, longest, seqs - 1)] + [longest]
    p = Pool(hq, lens, hkv, spread=0.7)
    for new, bit in ((rng.integers(0, 2, seqs), 0), ([1] * seqs, 0), ([0] * seqs, 0),
                     ([2] + [1] * (seqs - 2) + [0], _lib.PA_DEV_BAD_QUERY_LEN), ([1, 1, "bad"] + [1] * (seqs - 3), _lib.PA_DEV_BAD_CONTEXT_LEN)):
        counts = [0 if n == "bad" else int(n) for n in new]
        start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        total = int(start[-1])
        if "bad" in list(new):
            start[2] = -4                                    # sequences 1 and 2
        rows = [(b, lens[b] - 1) for b in range(seqs) if counts[b] == 1 and not ("bad" in list(new) and b in (1, 2))]
        at = [int(start[b]) for b, _ in rows]
        q = _query(p, total + 3, hq)
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = pkv.decode_block_fp8(q.cuda(), *p.device(), query_start=torch.from_numpy(start).cuda(), partition_size=partition,
                                   out=out, status=status)
        assert got is out and int(status.item()) == bit
        ref, bound = p.reference(q.double().numpy()[at], rows, D ** -0.5)
        _check(out[at], ref, bound, f"{bit}")
        rest = np.setdiff1d(np.arange(total + 3), at)
        assert (out[torch.from_numpy(rest).cuda()] == 7.0).all()


def test_decode_flags_bad_scales_tables_lengths_and_queries(pkv):
    from paged_kv_cache_100_gb300 import _lib
    lens = [40, 40]
    for what, bit in (("scale", _lib.PA_DEV_RANGE), ("zero", _lib.PA_DEV_RANGE), ("query", _lib.PA_DEV_RANGE),
                      ("table", _lib.PA_DEV_BAD_BLOCK_ID), ("length", _lib.PA_DEV_BAD_CONTEXT_LEN)):
        p = Pool(5, lens, 2, poison=False)
        q = _query(p, 2, 4)
        if what == "scale":
            p.vs[p.tables[1, 1]] = float("inf")
        if what == "zero":
            p.vs[p.tables[1, 1]] = 0.0
        if what == "query":
            q[1, 0, 0] = 70000.0
        dev = p.device()
        if what == "table":
            dev[4][1, 1] = p.blocks
        if what == "length":
            dev[5][1] = 16 * 3 + 1
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pkv.decode_block_fp8(q.cuda(), *dev, status=status)
        assert int(status.item()) == bit, what
        ref, bound = p.reference(q.double().numpy()[:1], [(0, 39)], D ** -0.5)
        _check(out[:1], ref, bound, what)                   # the other sequence is not touched by it


def test_decode_nan_code_reaches_the_output(pkv):
    p = Pool(6, [33, 20, 20], 1, poison=False)
    p.vc[p.tables[0, 1], 0, 3, 7] = 0x7F
    p.kc[p.tables[2, 0], 0, 3, 7] = 0x7F
    q = _query(p, 3, 2)
    out = pkv.decode_block_fp8(q.cuda(), *p.device()).cpu()
    assert torch.isnan(out[0, :, 7]).all() and torch.isfinite(out[0, :, :7]).all()
    assert torch.isfinite(out[1]).all() and torch.isnan(out[2]).all()


def test_decode_long_context_and_given_workspace(pkv):
    lens = [20000, 3]
    p = Pool(9, lens, 2, spread=0.7)
    q = _query(p, 2, 4)
    dev = p.device()
    for P in (0, 512, 16384):
        need = pkv.decode_block_fp8_workspace_bytes(2, 4, 2, D, p.tables.shape[1], P)
        ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
        out = pkv.decode_block_fp8(q.cuda(), *dev, partition_size=P, workspace=ws[:need])
        ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(lens)], D ** -0.5)
        _check(out, ref, bound, f"P={P}")
        assert (ws[need:] == 0xAB).all()


@pytest.mark.parametrize("longest", [20, 250, 500, 900])
@pytest.mark.parametrize("hq,hkv,window", [(2, 2, 0), (14, 2, 0), (6, 2, 120)])
def test_decode_cut_into_clusters(pkv, longest, hq, hkv, window):
    """Contexts that are cut into two, four and eight parts, and not at all."""
    lens = [min(n + 3 * i, longest) for i in range(2) for n in LENS] + [longest]
    p = Pool(longest + hq, lens, hkv, spread=0.7)
    q = _query(p, len(lens), hq)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((16,), 0xAB, dtype=torch.uint8, device="cuda")
    assert pkv.decode_block_fp8_workspace_bytes(len(lens), hq, hkv, D, p.tables.shape[1], 0, window) == 0
    out = pkv.decode_block_fp8(q.cuda(), *p.device(), window=window, status=status, workspace=ws)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(lens)], D ** -0.5, window)
    _check(out, ref, bound, f"{longest}")
    assert int(status.item()) == 0 and (ws == 0xAB).all()


@pytest.mark.parametrize("hq,hkv,window,partition", [(16, 16, 0, 0), (48, 16, 0, 0), (16, 16, 100, 0), (32, 16, 0, 64),
                                                     (11, 1, 30, 16)])
def test_decode_many_short_contexts(pkv, hq, hkv, window, partition):
    """More CTAs than the GPU holds, each with a short part: one warp per CTA."""
    lens = [(37 * i) % 256 for i in range(110)] + [256]
    p = Pool(hq + window + partition, lens, hkv, spread=0.7)
    q = _query(p, len(lens), hq)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.decode_block_fp8(q.cuda(), *p.device(), window=window, status=status, partition_size=partition)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(lens)], D ** -0.5, window)
    _check(out, ref, bound, f"{hq}/{hkv} W={window} P={partition}")
    assert (out[0] == 0).all() and int(status.item()) == 0


@pytest.mark.parametrize("lens,hq,hkv,window", [([777], 32, 8, 0), (LENS, 8, 2, 0), ([40, 2100, 0, 2048], 8, 8, 0),
                                                ([(37 * i) % 100 for i in range(80)], 8, 8, 0), ([(37 * i) % 100 for i in range(80)], 16, 8, 30),
                                                ([5, 300] * 70, 12, 4, 0)])
@pytest.mark.parametrize("width", [1000, 8192])
def test_decode_with_tables_wider_than_the_contexts(pkv, lens, hq, hkv, window, width):
    """Tables as wide as a model's limit, of which the contexts fill little: most parts of the grid are empty."""
    p = Pool(width + len(lens), lens, hkv, spread=0.7, width=width)
    q = _query(p, len(lens), hq)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.decode_block_fp8(q.cuda(), *p.device(), window=window, status=status)
    ref, bound = p.reference(q.double().numpy(), [(b, n - 1) for b, n in enumerate(lens)], D ** -0.5, window)
    _check(out, ref, bound, f"{width}")
    assert int(status.item()) == 0


@pytest.mark.parametrize("width", [700, 8192])
def test_prefill_with_tables_wider_than_the_contexts(pkv, width):
    for chunks, lens in (([5], [100]), ([16, 1, 40], [16, 333, 700])):
        p = Pool(width + len(lens), lens, 2, spread=0.7, width=width)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q, out, rows = _prefill(pkv, p, chunks, 8, status=status)
        ref, bound = p.reference(q.double().numpy(), rows, D ** -0.5, floor=4.0)
        _check(out, ref, bound, f"{width}")
        assert int(status.item()) == 0


def test_decode_graph_replay_and_streams(pkv):
    p = Pool(11, [900, 1, 2000, 64], 4)
    q = _query(p, 4, 16).cuda()
    dev = p.device()
    want = pkv.decode_block_fp8(q, *dev, partition_size=256)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pkv.decode_block_fp8(q, *dev, partition_size=256, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = pkv.decode_block_fp8(q, *dev, partition_size=256)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def _prefill(pkv, p, chunks, hq, window=0, scale=None, status=None, q=None, longest=None, **over):
    start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    q = _query(p, int(start[-1]), hq) if q is None else q
    out = pkv.prefill_block_fp8(q.cuda(), *p.device(), torch.from_numpy(start).cuda(), longest, scale, window=window,
                                status=status, **over)
    rows = [(b, int(p.lens[b]) - n + i) for b, n in enumerate(chunks) for i in range(n)]
    return q, out, rows


PREFILL = [  # chunks, lengths
    ([1], [1]), ([17], [17]), ([130], [200]), ([5, 1, 40], [5, 33, 300]), ([0, 64, 0, 3], [0, 64, 50, 131]),
    ([300], [700]), ([16, 128, 129], [16, 1000, 129])]


@pytest.mark.parametrize("chunks,lens", PREFILL)
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (8, 1), (16, 1)])
def test_prefill_matches(pkv, chunks, lens, hq, hkv):
    p = Pool(sum(chunks) + hq, lens, hkv)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, out, rows = _prefill(pkv, p, chunks, hq, status=status)
    ref, bound = p.reference(q.double().numpy(), rows, D ** -0.5, floor=4.0)
    _check(out, ref, bound, f"{hq}/{hkv}")
    assert int(status.item()) == 0


@pytest.mark.parametrize("window", [1, 15, 16, 100, 129, 1000])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 1)])
def test_prefill_window(pkv, window, hq, hkv):
    chunks, lens = [40, 1, 200], [40, 333, 700]
    p = Pool(window, lens, hkv)
    q, out, rows = _prefill(pkv, p, chunks, hq, window=window)
    ref, bound = p.reference(q.double().numpy(), rows, D ** -0.5, window, floor=4.0)
    _check(out, ref, bound, f"W={window}")


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 1)])
def test_prefill_rising_scores_and_scales(pkv, hq, hkv):
    """References that rise in later tiles, value scales over the whole range, key scales that are no
    powers of two, a negative softmax scale."""
    lens, chunks = [600, 400], [50, 400]
    p = Pool(21, lens, hkv, poison=False)
    p.vs[:] = torch.exp2(torch.randint(-32, 32, p.vs.shape, generator=p.g).float())
    p.ks[p.tables[0, :38]] *= torch.linspace(0.2, 60.0, 38)[:, None]
    p.vs[p.tables[1, :25]] = torch.rand(25, hkv, generator=p.g) + 0.1
    p.vs[p.tables[1, 13]] = 3.0e4
    for scale in (D ** -0.5, -0.02):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q, out, rows = _prefill(pkv, p, chunks, hq, scale=scale, status=status)
        pick = list(range(0, len(rows), 7))
        ref, bound = p.reference(q.double().numpy()[pick], [rows[i] for i in pick], scale, floor=4.0)
        _check(out[pick], ref, bound, f"scale {scale}")
        assert int(status.item()) == 0


def test_prefill_many_items(pkv):
    """More items than SMs, long and short chunks together; rows sampled."""
    rng = np.random.default_rng(0)
    chunks = [int(x) for x in rng.integers(1, 400, 12)] + [1] * 70
    lens = [c + int(x) for c, x in zip(chunks, rng.integers(0, 900, len(chunks)))]
    p = Pool(2, lens, 2, spread=0.7)
    q, out, rows = _prefill(pkv, p, chunks, 8, longest=max(chunks))
    pick = sorted(rng.choice(len(rows), 300, replace=False).tolist())
    ref, bound = p.reference(q.double().numpy()[pick], [rows[i] for i in pick], D ** -0.5, floor=4.0)
    _check(out[pick], ref, bound)


@pytest.mark.parametrize("hq,hkv", [(8, 1), (4, 2)])
@pytest.mark.parametrize("window", [0, 900])
def test_prefill_cut_along_the_context(pkv, hq, hkv, window):
    """Few rows over long contexts: items are cut into parts and merged, short sequences beside them not."""
    chunks, lens = [5, 70, 3, 0, 20], [3000, 2100, 3, 17, 900]
    p = Pool(hq + window, lens, hkv, spread=0.7)
    need = pkv.lib().pa_prefill_block_fp8_workspace_bytes(len(lens), hq, hkv, D, p.tables.shape[1], sum(chunks), 70, window)
    assert need > sum(chunks) * hq * D * 4 or window
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    q, out, rows = _prefill(pkv, p, chunks, hq, window=window, status=status, longest=70, workspace=ws[:need])
    ref, bound = p.reference(q.double().numpy(), rows, D ** -0.5, window, floor=4.0)
    _check(out, ref, bound, f"{hq}/{hkv}")
    assert (ws[need:] == 0xAB).all() and int(status.item()) == 0


def test_prefill_cut_into_more_parts_than_sms(pkv):
    """80 items of which the long ones are cut in three: CTAs take several parts each, by ticket."""
    lens = [6000, 3000, 1500] + [20 + 37 * i for i in range(37)]
    chunks = [1 + i % 7 for i in range(40)]
    p = Pool(21, lens, 2, spread=0.7)
    need = pkv.lib().pa_prefill_block_fp8_workspace_bytes(len(lens), 4, 2, D, p.tables.shape[1], sum(chunks), 7, 0)
    assert need > 2 * sum(chunks) * 4 * D * 4
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        q, out, rows = _prefill(pkv, p, chunks, 4, status=status, longest=7, workspace=ws[:need])
        ref, bound = p.reference(q.double().numpy(), rows, D ** -0.5, floor=4.0)
        _check(out, ref, bound)
    assert (ws[need:] == 0xAB).all() and int(status.item()) == 0


def test_prefill_flags(pkv):
    from paged_kv_cache_100_gb300 import _lib
    chunks, lens = [20, 30], [60, 40]
    for what, bit in (("scale", _lib.PA_DEV_RANGE), ("table", _lib.PA_DEV_BAD_BLOCK_ID),
                      ("length", _lib.PA_DEV_BAD_CONTEXT_LEN), ("longest", _lib.PA_DEV_BAD_QUERY_LEN)):
        p = Pool(5, lens, 2, poison=False)
        q = _query(p, 50, 4)
        longest = 30
        if what == "scale":
            p.vs[p.tables[1, 1]] = float("nan")
        if what == "table":
            p.tables[1, 0] = -7
        if what == "length":
            p.lens[1] = 29
        if what == "longest":
            longest = 20
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        _, out, rows = _prefill(pkv, p, chunks, 4, status=status, q=q, longest=longest)
        assert int(status.item()) == bit, what
        ref, bound = p.reference(q.double().numpy()[:20], rows[:20], D ** -0.5, floor=4.0)
        _check(out[:20], ref, bound, what)


@pytest.mark.parametrize("bad", [200, -5, 1 << 30])
@pytest.mark.parametrize("longest,blocks", [(30, None), (30, 400)])
def test_prefill_bad_start_entries_leave_other_sequences_alone(pkv, bad, longest, blocks):
    """An entry of query_start that falls or leaves the rows: its two sequences are flagged and not computed,
    those beside them are, with their contexts cut into parts or not."""
    from paged_kv_cache_100_gb300 import _lib
    chunks, lens = [20, 7, 11, 30, 5], [60, 5000 if blocks else 40, 3000 if blocks else 33, 2000 if blocks else 50, 1500 if blocks else 9]
    p = Pool(40, lens, 2, width=blocks, spread=0.7)
    start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    q = _query(p, int(start[-1]), 4)
    given = start.copy()
    given[2] = bad                                           # sequences 1 and 2
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.prefill_block_fp8(q.cuda(), *p.device(), torch.from_numpy(given).cuda(), longest, out=out, status=status)
    rows = [(b, lens[b] - n + i) for b, n in enumerate(chunks) for i in range(n)]
    pick = [i for i, (b, _) in enumerate(rows) if b in (0, 3, 4)]
    ref, bound = p.reference(q.double().numpy()[pick], [rows[i] for i in pick], D ** -0.5, floor=4.0)
    _check(out[pick], ref, bound, f"{bad}")
    assert (out[20:38] == 7.0).all() and int(status.item()) == _lib.PA_DEV_BAD_CONTEXT_LEN


def test_prefill_queries_of_any_size(pkv):
    """Rows of large, tiny and zero queries, a row with an outlier element, infinite and NaN elements."""
    p = Pool(15, [90], 2, spread=0.7)
    q = _query(p, 40, 8)
    q[3] = (q[3].float() * 2.0 ** 100).to(torch.bfloat16)
    q[4] = (q[4].float() * 2.0 ** -130).to(torch.bfloat16)
    q[5] = 0
    q[6, :, 17] = 40.0
    q[7, 2, 5], q[8, 3, 0] = float("inf"), float("nan")
    p.ks[:] = torch.where(torch.isnan(p.ks), p.ks, torch.full_like(p.ks, 2.0 ** -9))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, out, rows = _prefill(pkv, p, [40], 8, status=status, q=q)
    qd = q.double().numpy()
    bad = ~np.isfinite(qd).all(-1)
    qd[bad] = 0
    ref, bound = p.reference(qd, rows, D ** -0.5, floor=4.0)
    assert torch.isnan(out.cpu()[torch.from_numpy(bad)]).all()
    keep = ~bad
    keep[3] = False                                          # one-hot rows: the largest score alone decides
    got = out.double().cpu().numpy()
    err = np.abs(got - ref)[keep]
    assert (err <= (bound + 2.0 ** -8 * (np.abs(ref) + bound))[keep]).all()
    assert np.isfinite(got[3]).all() and int(status.item()) == 0


@pytest.mark.parametrize("hq,hkv,window,chunks,lens", [(4, 2, 0, [300, 40], [310, 700]), (8, 1, 70, [300, 40], [310, 700]),
                                                       (2, 2, 0, [12], [2100]), (32, 2, 900, [9], [2100]),
                                                       (8, 8, 0, [200] * 24, [200] * 24)])
def test_prefill_nan_values_reach_the_rows_that_attend_to_them(pkv, hq, hkv, window, chunks, lens):
    """A NaN code of V gives NaN in its column to the rows that attend to its position, and to no other:
    not to rows before it in its chunk, nor to rows whose window has passed it."""
    p = Pool(hq + window, lens, hkv, spread=0.7)
    nan = [(b, pos, h, d) for b, n in enumerate(lens)
           for pos, h, d in ((n - 2, 0, 3), (n - chunks[b] // 2, hkv - 1, 127), (n - chunks[b], 0, 64), (n // 3, 0, 5))][:24]
    for k, (b, pos, h, d) in enumerate(nan):
        p.vc[p.tables[b, pos // 16], h, pos % 16, d] = 0x7F if k % 2 else 0xFF
    q, out, rows = _prefill(pkv, p, chunks, hq, window=window)
    want = np.zeros((len(rows), hq, D), bool)
    group = hq // hkv
    for i, (b, last) in enumerate(rows):
        for bb, pos, h, d in nan:
            if bb == b and pos <= last and (window == 0 or pos > last - window):
                want[i, h * group:(h + 1) * group, d] = True
    got = out.double().cpu().numpy()
    assert want.any() and (np.isnan(got) == want).all()
    for b, pos, h, d in nan:
        p.vc[p.tables[b, pos // 16], h, pos % 16, d] = 0
    ref, bound = p.reference(q.double().numpy(), rows, D ** -0.5, window, floor=4.0)
    err = np.abs(got - ref)
    assert (err <= bound + 2.0 ** -8 * (np.abs(ref) + bound))[~want].all()


def test_prefill_leaves_rows_behind_the_last_sequence(pkv):
    p = Pool(8, [50], 1)
    q = _query(p, 64, 4)
    out = torch.full((64, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    pkv.prefill_block_fp8(q.cuda(), *p.device(), start, 50, out=out)
    ref, bound = p.reference(q.double().numpy()[:50], [(0, i) for i in range(50)], D ** -0.5, floor=4.0)
    _check(out[:50], ref, bound)
    assert (out[50:] == 7.0).all()


def test_prefill_graph_and_decode_agree(pkv):
    """A chunk of one token is a decode; a captured prefill replays the same bytes."""
    lens = [300, 17, 1000]
    p = Pool(31, lens, 2, spread=0.7)
    q = _query(p, 3, 8).cuda()
    dev = p.device()
    start = torch.arange(4, dtype=torch.int32, device="cuda")
    one = pkv.prefill_block_fp8(q, *dev, start, 1)
    ref, bound = p.reference(q.cpu().double().numpy(), [(b, n - 1) for b, n in enumerate(lens)], D ** -0.5, floor=4.0)
    _check(one, ref, bound)
    _check(pkv.decode_block_fp8(q, *dev), ref, bound)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = pkv.prefill_block_fp8(q, *dev, start, 1)
    for _ in range(2):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, one)


def test_pools_past_32_bits(pkv):
    """A pool of more than 2^32 bytes: writes, decode and prefill at its far end."""
    blocks, hkv, hq, n = 2_200_000, 1, 4, 70
    kc = torch.zeros(blocks, hkv, 16, D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = (torch.ones(blocks, hkv, device="cuda") for _ in range(2))
    assert kc.numel() > 1 << 32
    g = torch.Generator().manual_seed(1)
    table = torch.tensor([[blocks - 1, 3, blocks - 700, blocks - 2, 5]], dtype=torch.int32)
    x = torch.randn(n, 2 * hkv, D, generator=g).to(torch.bfloat16)
    pos = torch.arange(n)
    slots = table[0][pos // 16].long() * 16 + pos % 16
    xd = x.cuda()
    pkv.rope_cache_write(None, xd[:, :1], xd[:, 1:], None, None, kc, vc, slots.cuda(), k_scales=ks, v_scales=vs)
    small = torch.tensor([blocks - 1, 3, blocks - 700, blocks - 2, 5])
    kv, vv = R.decode_codes(kc[small.cuda()]), R.decode_codes(vc[small.cuda()])
    kss, vss = ks[small.cuda()].double().cpu().numpy(), vs[small.cuda()].double().cpu().numpy()
    for got, ref in ((kv * kss[:, :, None, None], x[:, 0]), (vv * vss[:, :, None, None], x[:, 1])):
        rows = got[:, 0].reshape(80, D)[:n]
        assert (np.abs(rows - ref.double().numpy()) <= 2.0 ** -4 * np.abs(ref.double().numpy()) + 2.0 ** -10 * kss.max()).all()
    assert int(kc.view(torch.int64).count_nonzero()) <= n * D // 8        # nothing else was written
    q = torch.randn(3, hq, D, generator=g).to(torch.bfloat16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    args = (kc, vc, ks, vs, table.cuda(), lens)
    start = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    order = np.arange(5)
    for rows, out in (([n - 1], pkv.decode_block_fp8(q[2:].cuda(), *args)), ([n - 3, n - 2, n - 1], pkv.prefill_block_fp8(q.cuda(), *args, start, 3))):
        for i, last in enumerate(rows):
            qq = q[2 if len(rows) == 1 else i].double().numpy()
            ref, bound = R.attention(qq, kv[:, 0], kss[:, 0], vv[:, 0], vss[:, 0], order, 0, last + 1, D ** -0.5, floor=4.0)
            _check(out[i], ref, bound)


@pytest.mark.parametrize("window", [0, 300])
def test_prefill_nan_values_beside_many_short_chunks(pkv, window):
    """More items than SMs, of which those with two tiles of rows hold NaN codes and most others have one
    tile: the NaNs stay with the rows that attend to them, and no wait gives up."""
    hq, hkv = 16, 2                                          # 16 tokens a tile
    rng = np.random.default_rng(window)
    chunks = [40 if i % 20 == 0 else 1 + i % 3 for i in range(240)]
    lens = [n + int(x) for n, x in zip(chunks, rng.integers(0, 120, len(chunks)))]
    lens[0] = lens[100] = 2500
    p = Pool(77 + window, lens, hkv, spread=0.7)
    nan = [(b, pos, b // 20 % hkv, 5 * (b % 25)) for b in range(0, 240, 20) for pos in (lens[b] - 2, lens[b] - 30, lens[b] // 2)]
    for k, (b, pos, h, d) in enumerate(nan):
        p.vc[p.tables[b, pos // 16], h, pos % 16, d] = 0x7F if k % 2 else 0xFF
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, out, rows = _prefill(pkv, p, chunks, hq, window=window, status=status, longest=40)
    want = np.zeros((len(rows), hq, D), bool)
    for i, (b, last) in enumerate(rows):
        for bb, pos, h, d in nan:
            if bb == b and pos <= last and (window == 0 or pos > last - window):
                want[i, h * hq // hkv:(h + 1) * hq // hkv, d] = True
    got = out.double().cpu().numpy()
    assert want.any() and (np.isnan(got) == want).all()
    assert int(status.item()) == 0
    for b, pos, h, d in nan:
        p.vc[p.tables[b, pos // 16], h, pos % 16, d] = 0
    pick = sorted(rng.choice(len(rows), 250, replace=False).tolist())
    ref, bound = p.reference(q.double().numpy()[pick], [rows[i] for i in pick], D ** -0.5, window, floor=4.0)
    err = np.abs(got[pick] - ref)
    assert (err <= bound + 2.0 ** -8 * (np.abs(ref) + bound))[~want[pick]].all()


@pytest.mark.parametrize("window", [0, 50000])
def test_prefill_nan_values_in_long_contexts(pkv, window):
    """NaN codes at a long context's beginning and end, in steps that all rows attend to and in the steps of
    the diagonal and of the window's start: each reaches the rows that attend to it, and no wait gives up."""
    hq, hkv, chunk, length = 8, 1, 40, 60000
    p = Pool(5 + window, [length, 100], hkv, spread=0.7)
    nan = [(pos, d) for d, pos in enumerate((3, 130, length // 2, length - 45, length - 30, length - 2, length - 50000 - 1,
                                             length - 50000 - 20, length - 50000 + 7))] + [(length - 9, 127), (length - 9, 64)]
    for pos, d in nan:
        p.vc[p.tables[0, pos // 16], 0, pos % 16, d] = 0x7F
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, out, rows = _prefill(pkv, p, [chunk, 7], hq, window=window, status=status, longest=chunk)
    want = np.zeros((len(rows), hq, D), bool)
    for i, (b, last) in enumerate(rows):
        for pos, d in nan:
            if b == 0 and pos <= last and (window == 0 or pos > last - window):
                want[i, :, d] = True
    assert (np.isnan(out.double().cpu().numpy()) == want).all() and int(status.item()) == 0
