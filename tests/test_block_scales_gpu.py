"""Scales of block-scaled pools go where their blocks go: copy-on-write copies and swaps."""
import numpy as np
import pytest
import torch

from tests import block8_ref as R

pytestmark = pytest.mark.gpu
D, HQ = 128, 8


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_100_gb300.build import build
    build()
    import paged_kv_cache_100_gb300 as m
    return m


def _pools(seed, blocks, hkv, dim=D):
    g = torch.Generator().manual_seed(seed)
    kc, ks = R.pools(g, blocks, hkv, dim, 3.0)
    vc, vs = R.pools(g, blocks, hkv, dim, 3.0)
    return [t.cuda() for t in (kc, vc, ks, vs)]


@pytest.mark.parametrize("hkv,dim", [(1, 16), (3, 128), (40, 64), (300, 16)])
def test_block_copy_takes_the_scales(pkv, hkv, dim):
    from paged_kv_cache_100_gb300 import _lib
    kc, vc, ks, vs = _pools(hkv, 12, hkv, dim)
    before = [t.clone() for t in (kc, vc, ks, vs)]
    # two copies of one source; then an index outside, a copy onto itself, and two of one destination
    pairs = torch.tensor([[3, 7], [3, 0], [12, 1], [5, 5], [2, 9], [4, 9]], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.block_copy(kc, vc, pairs, k_scales=ks, v_scales=vs, status=status)
    for t, old in zip((kc, vc, ks, vs), before):
        want = old.clone()
        want[7], want[0] = old[3], old[3]
        assert torch.equal(t, want)
    assert int(status.item()) == _lib.PA_DEV_BAD_COPY_PAIR


@pytest.mark.parametrize("where", ["host", "device"])
@pytest.mark.parametrize("hkv,dim", [(2, 128), (260, 16)])
def test_swap_takes_the_scales(pkv, where, hkv, dim):
    from paged_kv_cache_100_gb300 import _lib
    kc, vc, ks, vs = _pools(hkv + 1, 10, hkv, dim)
    before = [t.clone() for t in (kc, vc, ks, vs)]
    ids = torch.tensor([8, 1, 4], dtype=torch.int32, device="cuda")
    given = {}
    if where == "device":
        given = dict(staging=torch.empty(3, 2, hkv, 16, dim, dtype=torch.uint8, device="cuda"),
                     scale_staging=torch.empty(3, 2, hkv, device="cuda"))
    staging, scales = pkv.swap_out(kc, vc, ids, k_scales=ks, v_scales=vs, **given)
    torch.cuda.synchronize()
    assert scales.shape == (3, 2, hkv) and scales.is_cuda == (where == "device")
    assert torch.equal(scales[:, 0].cuda(), ks[ids.long()]) and torch.equal(scales[:, 1].cuda(), vs[ids.long()])
    for t in (kc, vc):
        t.fill_(0x7F)
    for t in (ks, vs):
        t.fill_(float("nan"))
    back = torch.tensor([0, 9, 10, 6][:3], dtype=torch.int32, device="cuda")          # the third lies outside
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.swap_in(kc, vc, back, staging, k_scales=ks, v_scales=vs, scale_staging=scales, status=status)
    for t, old in zip((kc, vc, ks, vs), before):
        assert torch.equal(t[0], old[8]) and torch.equal(t[9], old[1])
    assert torch.isnan(ks[1:9]).all() and (kc[1:9] == 0x7F).all() and int(status.item()) == _lib.PA_DEV_BAD_BLOCK_ID


def test_forked_and_preempted_sequences(pkv):
    """A fork that diverges in a shared, part-filled block (copy-on-write, then a larger row that raises the copy's
    scale), and a sequence that is swapped out, its blocks written over, and back in."""
    hkv, blocks, width = 2, 30, 6
    g = torch.Generator().manual_seed(4)
    bm = pkv.BlockManager(blocks)
    kc, vc, ks, vs = _pools(1, blocks, hkv)
    for t in (ks, vs):
        t.fill_(2.0 ** 20)                                   # whatever other requests left there
    scales = dict(k_scales=ks, v_scales=vs)
    lens = {0: 37, 1: 70}
    truth = {}

    def write(seq, first, n, size):
        x = (torch.randn(n, 2 * hkv, D, generator=g) * size).to(torch.bfloat16)
        table = np.array(bm.table(seq))
        pos = np.arange(first, first + n)
        slots = torch.from_numpy(table[pos // 16].astype(np.int64) * 16 + pos % 16).cuda()
        d = x.cuda()
        pkv.rope_cache_write(None, d[:, :hkv], d[:, hkv:], None, None, kc, vc, slots, **scales)
        truth.setdefault(seq, []).extend(x.double().numpy())

    for seq, n in lens.items():
        bm.alloc_seq(seq, n)
        write(seq, 0, n, 1.0)
    bm.fork(0, 2)
    truth[2] = list(truth[0])
    lens[2] = lens[0]
    _, cow = bm.append_slot(2)
    assert cow is not None
    pkv.block_copy(kc, vc, torch.tensor([cow], dtype=torch.int32, device="cuda"), **scales)
    write(2, 37, 1, 64.0)
    lens[2] = 38

    def check():
        q = torch.randn(3, HQ, D, generator=g).to(torch.bfloat16)
        tables, lengths = bm.fill_tables([0, 1, 2], width)
        out = pkv.decode_block_fp8(q.cuda(), kc, vc, ks, vs, torch.from_numpy(tables).cuda(), torch.from_numpy(lengths).cuda())
        kv, vv = R.decode_codes(kc), R.decode_codes(vc)
        kss, vss = ks.double().cpu().numpy(), vs.double().cpu().numpy()
        for seq in range(3):
            for t in range(lens[seq]):                       # what the pools hold is what was written, to half a code step
                blk = tables[seq, t // 16]
                for vals, sc, col in ((kv, kss, slice(0, hkv)), (vv, vss, slice(hkv, None))):
                    want = truth[seq][t][col]
                    got = vals[blk, :, t % 16] * sc[blk][:, None]
                    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * sc[blk][:, None]).all(), (seq, t)
            for h in range(hkv):
                j = slice(h * HQ // hkv, (h + 1) * HQ // hkv)
                ref, bound = R.attention(q[seq, j].double().numpy(), kv[:, h], kss[:, h], vv[:, h], vss[:, h], tables[seq], 0,
                                         lens[seq], D ** -0.5)
                err = np.abs(out[seq, j].double().cpu().numpy() - ref)
                assert (err <= bound + 2.0 ** -8 * (np.abs(ref) + bound)).all()

    check()
    gone = bm.swap_out(1)
    staging, staged = pkv.swap_out(kc, vc, torch.tensor(gone, dtype=torch.int32, device="cuda"), **scales)
    bm.alloc_seq(3, 16 * len(gone))
    write(3, 0, 16 * len(gone), 2.0 ** 12)
    back = bm.swap_in(1)
    pkv.swap_in(kc, vc, torch.tensor(back, dtype=torch.int32, device="cuda"), staging, scale_staging=staged, **scales)
    check()
