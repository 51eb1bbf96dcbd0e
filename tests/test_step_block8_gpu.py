"""The step operators run together, as a serving loop would: plan the step on the GPU, turn and write
its rows into block-scaled pools, attend (a prefill of ragged prompts, then decode steps), all from
device-resident state; checked against 64-bit arithmetic on the values the pools hold, and against a
captured graph of the same step."""
import numpy as np
import pytest
import torch

from tests import block8_ref as R

pytestmark = pytest.mark.gpu
D, HQ, HKV = 128, 8, 2


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_100_gb300.build import build
    build()
    import paged_kv_cache_100_gb300 as m
    return m


class Serving:
    """Device state of a batch: pools, scales, tables, lengths and the free stack."""

    def __init__(self, pkv, seqs, blocks, width):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pkv, self.blocks = pkv, blocks
        self.kc = torch.full((blocks, HKV, 16, D), 0x7F, dtype=torch.uint8, device="cuda")
        self.vc = self.kc.clone()
        self.ks = torch.full((blocks, HKV), float("nan"), device="cuda")
        self.vs = self.ks.clone()
        self.tables = torch.full((seqs, width), -1, **i32)
        self.lens = torch.zeros(seqs, **i32)
        self.free = torch.randperm(blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.num_free = torch.tensor([blocks], **i32)
        self.status = torch.zeros(1, **i32)
        self.rope = pkv.rotary_plan(D, 10000.0)

    def step(self, qkv, new, longest):
        """qkv [capacity][HQ + 2 HKV][D]; returns the attention's output and the plan."""
        pkv = self.pkv
        p = pkv.plan_step(self.tables, self.lens, new, self.free, self.num_free, qkv.shape[0], self.blocks, status=self.status)
        q = pkv.rope_cache_write(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], p.positions, self.rope, self.kc,
                                 self.vc, p.slot_mapping, k_scales=self.ks, v_scales=self.vs, status=self.status)
        args = (self.kc, self.vc, self.ks, self.vs, self.tables, p.context_lens)
        if longest == 1:
            out = pkv.decode_block_fp8(q, *args, status=self.status)
        else:
            out = pkv.prefill_block_fp8(q, *args, p.query_start, longest, status=self.status)
        return out, q, p


def _check(s, out, q, p, new):
    tables, lens = s.tables.cpu().numpy(), p.context_lens.cpu().numpy()
    kv, vv = R.decode_codes(s.kc), R.decode_codes(s.vc)
    ks, vs = s.ks.double().cpu().numpy(), s.vs.double().cpu().numpy()
    qd, got = q.double().cpu().numpy(), out.double().cpu().numpy()
    row = 0
    for b, n in enumerate(new):
        for i in range(n):
            for h in range(HKV):
                j = slice(h * HQ // HKV, (h + 1) * HQ // HKV)
                ref, bound = R.attention(qd[row, j], kv[:, h], ks[:, h], vv[:, h], vs[:, h], tables[b], 0,
                                         lens[b] - n + i + 1, D ** -0.5, floor=4.0)
                err = np.abs(got[row, j] - ref)
                assert (err <= bound + 2.0 ** -8 * (np.abs(ref) + bound)).all(), (b, i, h)
            row += 1


def test_serving_steps(pkv):
    seqs, blocks, width = 6, 64, 12
    s = Serving(pkv, seqs, blocks, width)
    g = torch.Generator().manual_seed(3)
    prompts = [33, 1, 100, 16, 0, 47]
    truth_k, truth_v = [[] for _ in range(seqs)], [[] for _ in range(seqs)]

    def rows(n):
        return torch.randn(n, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16)

    def note(x, p, new):
        pos = p.positions.cpu().numpy()
        cos, sin = R.rotary_angles(pos, D)
        k, _ = R.rotate(x[:, HQ:HQ + HKV].double().numpy(), cos, sin, False)
        at = 0
        for b, n in enumerate(new):
            truth_k[b] += list(k[at:at + n])
            truth_v[b] += list(x[at:at + n, HQ + HKV:].double().numpy())
            at += n

    total = sum(prompts)
    x = rows(total + 5)                                     # five padded rows
    out, q, p = s.step(x.cuda(), torch.tensor(prompts, dtype=torch.int32, device="cuda"), max(prompts))
    _check(s, out, q, p, prompts)
    note(x, p, prompts)
    s.lens, s.num_free = p.context_lens, p.num_free
    for _ in range(20):
        x = rows(seqs)
        out, q, p = s.step(x.cuda(), torch.ones(seqs, dtype=torch.int32, device="cuda"), 1)
        _check(s, out, q, p, [1] * seqs)
        note(x, p, [1] * seqs)
        s.lens, s.num_free = p.context_lens, p.num_free
    assert int(s.status.item()) == 0
    # what the pools hold is the tokens' keys and values: a code is off by half a step (2^-4), and by
    # at most half a step more for each time its block's scale grew (subnormal codes: 2^-10 of the scale)
    lens, tables = s.lens.cpu().numpy(), s.tables.cpu().numpy()
    assert lens.tolist() == [n + 20 for n in prompts]
    used = [t for b in range(seqs) for t in tables[b, :-(-int(lens[b]) // 16)].tolist()]
    assert len(set(used)) == len(used) and int(s.num_free.item()) == blocks - len(used)
    for codes, scales, truth in ((s.kc, s.ks, truth_k), (s.vc, s.vs, truth_v)):
        v, sc = R.decode_codes(codes), scales.double().cpu().numpy()
        for b in range(seqs):
            for t in range(int(lens[b])):
                blk = tables[b, t // 16]
                got = v[blk, :, t % 16] * sc[blk][:, None]
                assert (np.abs(got - truth[b][t]) <= 2.0 ** -4 * np.abs(truth[b][t]) + 2.0 ** -9 * sc[blk][:, None]).all()


def test_captured_decode_step_replays(pkv):
    """One decode step captured with its two sets of lengths and counts, replayed for ten steps, equals
    the same steps called directly."""
    seqs, blocks, width = 5, 40, 6
    g = torch.Generator().manual_seed(5)
    xs = [torch.randn(seqs, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16).cuda() for _ in range(10)]
    one = torch.ones(seqs, dtype=torch.int32, device="cuda")
    a, b = Serving(pkv, seqs, blocks, width), Serving(pkv, seqs, blocks, width)
    direct = []
    for x in xs:
        out, _, p = a.step(x, one, 1)
        direct.append(out.clone())
        a.lens, a.num_free = p.context_lens, p.num_free
    x = xs[0].clone()
    lens, num_free = b.lens, b.num_free
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, p = b.step(x, one, 1)
        lens.copy_(p.context_lens)
        num_free.copy_(p.num_free)
    for i in range(10):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, direct[i]), i
    assert torch.equal(a.tables, b.tables) and torch.equal(a.kc, b.kc) and torch.equal(a.vc, b.vc)
    assert int(a.status.item()) == 0 and int(b.status.item()) == 0


def test_steps_in_which_some_sequences_bring_nothing(pkv):
    """Decode steps of a padded batch: idle sequences, and one whose table is full (it is passed over and flagged),
    move the others' rows in the flat list; query_start says where they are."""
    from paged_kv_cache_100_gb300 import _lib
    seqs, blocks, width = 7, 64, 3
    s = Serving(pkv, seqs, blocks, width)
    g = torch.Generator().manual_seed(9)
    prompts = [20, 0, 48, 17, 3, 30, 9]                      # the third one's table is full
    x = torch.randn(sum(prompts), HQ + 2 * HKV, D, generator=g).to(torch.bfloat16)
    out, q, p = s.step(x.cuda(), torch.tensor(prompts, dtype=torch.int32, device="cuda"), max(prompts))
    s.lens, s.num_free = p.context_lens, p.num_free
    for step in range(4):
        new = [int(b % 3 != step % 3) for b in range(seqs)]
        taken = [n if not (b == 2 and n) else 0 for b, n in enumerate(new)]
        x = torch.randn(seqs, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16).cuda()
        s.status.zero_()
        p = pkv.plan_step(s.tables, s.lens, torch.tensor(new, dtype=torch.int32, device="cuda"), s.free, s.num_free, seqs, blocks,
                          status=s.status)
        q = pkv.rope_cache_write(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], p.positions, s.rope, s.kc, s.vc, p.slot_mapping,
                                 k_scales=s.ks, v_scales=s.vs, status=s.status)
        out = pkv.decode_block_fp8(q, s.kc, s.vc, s.ks, s.vs, s.tables, p.context_lens, query_start=p.query_start, status=s.status)
        assert int(s.status.item()) == (_lib.PA_DEV_BAD_CONTEXT_LEN if new[2] else 0)
        assert p.query_start.tolist() == [0] + np.cumsum(taken).tolist()
        _check(s, out, q, p, taken)
        s.lens, s.num_free = p.context_lens, p.num_free
