"""A serving step over pools held in 4 bits, run together: plan on the GPU, turn and write its rows,
attend (a prefill of ragged prompts, then decode steps, then a chunk on what is cached); checked against
64-bit arithmetic, as captured graphs, on streams of their own and with several graphs at once."""
import numpy as np
import pytest
import torch

from tests import block8_ref as R
from tests import fp4_ref as F

pytestmark = pytest.mark.gpu
D, HQ, HKV = 128, 8, 2


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_100_gb300.build import build
    build()
    import paged_kv_cache_100_gb300 as m
    return m


class Serving:
    """Device state of a batch; the pools begin with NaN scales everywhere."""

    def __init__(self, pkv, seqs, blocks, width):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pkv, self.blocks = pkv, blocks
        self.kc, self.vc = pkv.fp4_pool(blocks, HKV, D).fill_(0xFF), pkv.fp4_pool(blocks, HKV, D).fill_(0xFF)
        self.tables = torch.full((seqs, width), -1, **i32)
        self.lens = torch.zeros(seqs, **i32)
        self.free = torch.randperm(blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.num_free = torch.tensor([blocks], **i32)
        self.status = torch.zeros(1, **i32)
        self.rope = pkv.rotary_plan(D, 10000.0)

    def step(self, qkv, new, longest, stream=None):
        """qkv [capacity][HQ + 2 HKV][D]; returns the attention's output, the turned queries and the plan."""
        pkv, how = self.pkv, dict(status=self.status, stream=stream)
        p = pkv.plan_step(self.tables, self.lens, new, self.free, self.num_free, qkv.shape[0], self.blocks, **how)
        q = pkv.rope_cache_write_fp4(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], p.positions, self.rope, self.kc,
                                     self.vc, p.slot_mapping, **how)
        args = (q, self.kc, self.vc, self.tables, p.context_lens)
        if longest == 1:
            out = pkv.decode_fp4(*args, query_start=p.query_start, **how)
        else:
            out = pkv.prefill_fp4(*args, p.query_start, longest, **how)
        return out, q, p


def _check(s, out, q, p, new):
    tables, lens = s.tables.cpu().numpy(), p.context_lens.cpu().numpy()
    kv, vv = F.unpack(s.kc)[2], F.unpack(s.vc)[2]
    one = np.ones(s.blocks)
    qd, got = q.double().cpu().numpy(), out.double().cpu().numpy()
    row = 0
    for b, n in enumerate(new):
        for i in range(n):
            for h in range(HKV):
                j = slice(h * HQ // HKV, (h + 1) * HQ // HKV)
                ref, bound = R.attention(qd[row, j], kv[:, h], one, vv[:, h], one, tables[b], 0, lens[b] - n + i + 1, D ** -0.5,
                                         floor=4.0)
                err = np.abs(got[row, j] - ref)
                assert (err <= bound + 2.0 ** -8 * (np.abs(ref) + bound)).all(), (b, i, h)
            row += 1


def test_serving_steps(pkv):
    seqs, blocks, width = 6, 64, 12
    s = Serving(pkv, seqs, blocks, width)
    g = torch.Generator().manual_seed(3)
    prompts, chunk = [33, 1, 100, 16, 0, 47], [5, 1, 0, 20, 3, 1]
    truth_k, truth_v = [[] for _ in range(seqs)], [[] for _ in range(seqs)]

    def run(new, spare):
        x = torch.randn(sum(new) + spare, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16)      # padded rows behind
        out, q, p = s.step(x.cuda(), torch.tensor(new, dtype=torch.int32, device="cuda"), max(new))
        _check(s, out, q, p, new)
        cos, sin = R.rotary_angles(p.positions.cpu().numpy(), D)
        k, _ = R.rotate(x[:, HQ:HQ + HKV].double().numpy(), cos, sin, False)
        at = 0
        for b, n in enumerate(new):
            truth_k[b] += list(k[at:at + n])
            truth_v[b] += list(x[at:at + n, HQ + HKV:].double().numpy())
            at += n
        s.lens, s.num_free = p.context_lens, p.num_free

    run(prompts, 5)
    for i in range(20):
        run([int(b % 3 != i % 3) for b in range(seqs)], i % 2)         # some sequences bring nothing
    run(chunk, 0)
    assert int(s.status.item()) == 0
    # what the pools hold is the tokens' keys and values, encoded: read back through the operator
    lens = s.lens.cpu().numpy()
    k, v = pkv.cache_read_fp4(s.kc, s.vc, s.tables, s.lens, dtype=torch.float32)
    for got, truth in ((k, truth_k), (v, truth_v)):
        got = got.double().cpu().numpy().reshape(seqs, width, HKV, 16, D)
        for b in range(seqs):
            assert len(truth[b]) == lens[b]
            if not truth[b]:
                continue
            rows = np.stack(truth[b])
            code, byte = F.encode(rows)
            want = F.values_of(code, byte)
            have = np.stack([got[b, t // 16, :, t % 16] for t in range(lens[b])])
            step = np.repeat(F.scales_of(byte), 16, -1)                # R.rotary_angles is not the plan's own angle:
            assert (np.abs(have - want) <= 2 * step).all() and (have != want).mean() < 1e-4     # borders may fall either way


def test_captured_decode_step_replays(pkv):
    """A decode step captured with its two sets of lengths and counts, replayed for ten steps, equals the
    same steps called directly; two graphs with workspaces of their own pools take turns."""
    seqs, blocks, width = 5, 40, 6
    g = torch.Generator().manual_seed(5)
    xs = [torch.randn(seqs, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16).cuda() for _ in range(10)]
    one = torch.ones(seqs, dtype=torch.int32, device="cuda")
    a = Serving(pkv, seqs, blocks, width)
    direct = []
    for x in xs:
        out, _, p = a.step(x, one, 1)
        direct.append(out.clone())
        a.lens, a.num_free = p.context_lens, p.num_free
    graphs = []
    for _ in range(2):
        b = Serving(pkv, seqs, blocks, width)
        x = xs[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, _, p = b.step(x, one, 1)
            b.lens.copy_(p.context_lens)
            b.num_free.copy_(p.num_free)
        graphs.append((graph, b, x, out))
    for i in range(10):
        for graph, b, x, out in graphs:
            x.copy_(xs[i])
            graph.replay()
        torch.cuda.synchronize()
        for graph, b, x, out in graphs:
            assert torch.equal(out, direct[i]), i
    for _, b, _, _ in graphs:
        assert torch.equal(a.tables, b.tables) and torch.equal(a.kc, b.kc) and torch.equal(a.vc, b.vc)
        assert int(b.status.item()) == 0


@pytest.mark.parametrize("lens,new", [([300, 40, 129], [64, 40, 1])])
def test_captured_prefill_and_split_decode_replay(pkv, lens, new):
    p = F.Batch(5, lens, HKV, D)
    dev = p.device()
    q = p.query(sum(new), HQ).cuda()
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    want = pkv.prefill_fp4(q, *dev, start, max(new))
    rows = q[:3].contiguous()
    want_d = pkv.decode_fp4(rows, *dev, partition_size=64)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = pkv.prefill_fp4(q, *dev, start, max(new))
            out_d = pkv.decode_fp4(rows, *dev, partition_size=64)
        graphs.append((graph, out, out_d))
    for graph, _, _ in graphs * 2:
        graph.replay()
    torch.cuda.synchronize()
    for _, out, out_d in graphs:
        assert torch.equal(out, want) and torch.equal(out_d, want_d)


def test_given_streams(pkv):
    """Work on a stream that is not the current one follows what that stream holds, output allocated for it."""
    p = F.Batch(7, [500, 77], HKV, D)
    dev = p.device()
    q = p.query(2, HQ).cuda()
    want = pkv.decode_fp4(q, *dev, partition_size=64)
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    want_p = pkv.prefill_fp4(q, *dev, start, 1)
    want_k, want_v = pkv.cache_read_fp4(*dev, key_out=torch.zeros(64, HKV, 16, D, device="cuda"),
                                        value_out=torch.zeros(64, HKV, 16, D, device="cuda"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late = torch.zeros_like(q)
    ko, vo = torch.zeros_like(want_k), torch.zeros_like(want_v)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
    outs = [(pkv.decode_fp4(late, *dev, partition_size=64, stream=side), pkv.prefill_fp4(late, *dev, start, 1, stream=side))
            for _ in range(3)]
    pkv.cache_read_fp4(*dev, key_out=ko, value_out=vo, stream=side)
    side.synchronize()
    for d, f in outs:
        assert torch.equal(d, want) and torch.equal(f, want_p)
    assert torch.equal(ko, want_k) and torch.equal(vo, want_v)


@pytest.mark.parametrize("kind", ["bf16", "block_fp8", "fp4"])
def test_longest_chunk_is_read_on_the_given_stream(pkv, kind):
    """max_query_len omitted: query_start may be what the given stream has yet to write."""
    p = F.Batch(7, [500, 77], HKV, D, poison=False)
    kc, vc, tables, lens = p.device()
    args = (kc, vc, tables, lens)
    call = pkv.prefill_fp4
    if kind != "fp4":
        k, v = (torch.from_numpy(F.unpack(t)[2]).to(torch.bfloat16).cuda() for t in (p.kc, p.vc))
        args, call = (k, v, tables, lens), pkv.prefill
    if kind == "block_fp8":
        one = torch.ones(p.blocks, HKV, device="cuda")
        args, call = (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), one, one, tables, lens), pkv.prefill_block_fp8
    q = p.query(25, HQ).cuda()
    start = torch.tensor([0, 20, 25], dtype=torch.int32, device="cuda")
    want = call(q, *args, start)                                     # (loads every kernel that the second call takes)
    late = torch.zeros_like(start)
    out = torch.full_like(want, 5.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        late.copy_(start)
    call(q, *args, late, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_calls_from_several_threads(pkv):
    """Calls of different sizes from threads with streams of their own."""
    import threading
    cases = []
    for seed, (lens, hq, hkv, dim) in enumerate([([3000, 10], 8, 8, 128), ([100] * 40, 16, 2, 128), ([900], 4, 4, 64), ([60] * 300, 8, 8, 256)]):
        p = F.Batch(seed, lens, hkv, dim)
        dev, q = p.device(), p.query(len(lens), hq).cuda()
        cases.append((q, dev, pkv.decode_fp4(q, *dev)))
    torch.cuda.synchronize()
    wrong = []

    def work(q, dev, want):
        stream = torch.cuda.Stream()
        for _ in range(20):
            out = pkv.decode_fp4(q, *dev, stream=stream)
            stream.synchronize()
            if not torch.equal(out, want):
                wrong.append(q.shape)

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
