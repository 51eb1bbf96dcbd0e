"""pa_plan_step: block tables, slots and positions on the GPU against a sequence-by-sequence model
and against the host block manager."""
import numpy as np
import pytest
import torch

from tests import block8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_100_gb300.build import build
    build()
    import paged_kv_cache_100_gb300 as m
    return m


def _run(pkv, tables, lens, new, free, num_free, cap, blocks, out=None, status=None):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    t = d(tables)
    p = pkv.plan_step(t, d(lens), d(new), d(free), d(np.array([num_free], np.int32)), cap, blocks, out=out, status=status)
    torch.cuda.synchronize()
    h = lambda x: x.cpu().numpy()  # noqa: E731
    return h(t), h(p.context_lens), h(p.query_start), h(p.slot_mapping), h(p.positions), int(p.num_free.item())


def _case(rng, B, hi, chunk, chunked):
    lens = rng.integers(0, hi + 1, B).astype(np.int32)
    new = np.where(rng.random(B) < chunked, rng.integers(0, chunk + 1, B), 1).astype(np.int32)
    have = -(-lens // 16)
    need = -(-(lens + new) // 16) - have
    width = int((-(-(lens + new) // 16)).max()) + 1
    perm = rng.permutation(int(have.sum() + need.sum()) + 5).astype(np.int32)
    tables = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        tables[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    return lens, new, tables, perm[at:], perm.size


def _same(got, want):
    for name, g, w in zip(("tables", "lens", "start", "slots", "positions", "free"), got, want):
        assert np.array_equal(g, w), name


@pytest.mark.parametrize("B,hi,chunk,chunked,slack", [
    (1, 0, 1, 1.0, 0), (1, 15, 1, 0.0, 0), (1, 100, 5000, 1.0, 7), (3, 40, 33, 0.5, 1), (64, 2048, 1, 0.0, 0),
    (257, 500, 64, 0.3, 100), (1024, 100, 3, 0.2, 0), (1025, 64, 20, 0.5, 3), (5000, 300, 40, 0.1, 50)])
def test_plan_matches_model(pkv, B, hi, chunk, chunked, slack):
    rng = np.random.default_rng(B + chunk)
    lens, new, tables, free, blocks = _case(rng, B, hi, chunk, chunked)
    cap = int(new.sum()) + slack
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(pkv, tables, lens, new, free, free.size, cap, blocks, status=status)
    _same(got, R.plan(tables, lens, new, free, free.size, cap, blocks))
    assert int(status.item()) == 0


@pytest.mark.parametrize("short", ["blocks", "tokens"])
@pytest.mark.parametrize("B", [5, 64, 2500])
def test_plan_stops_where_blocks_or_tokens_end(pkv, B, short):
    from paged_kv_cache_100_gb300 import _lib
    rng = np.random.default_rng(B)
    lens, new, tables, free, blocks = _case(rng, B, 100, 40, 0.7)
    new[B // 2:] = np.maximum(new[B // 2:], 17)
    width = int((-(-(lens + new) // 16)).max())
    tables = np.pad(tables, ((0, 0), (0, max(0, width - tables.shape[1]))), constant_values=-1)
    total = int(new.sum())
    cap = total * 2 // 3 if short == "tokens" else total
    nf = free.size if short == "tokens" else free.size // 2
    if short == "tokens":
        free = np.concatenate([free, np.arange(blocks, blocks + total, dtype=np.int32)])
        blocks, nf = blocks + total, free.size
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(pkv, tables, lens, new, free, nf, cap, blocks, status=status)
    _same(got, R.plan(tables, lens, new, free, nf, cap, blocks))
    assert int(status.item()) == _lib.PA_DEV_NO_BLOCKS


def test_plan_passes_over_bad_sequences_and_flags_bad_blocks(pkv):
    from paged_kv_cache_100_gb300 import _lib
    lens = np.array([3, -1, 20, 16, 30], np.int32)
    new = np.array([2, 4, -5, 40, 3], np.int32)             # the fourth does not fit its table
    tables = np.array([[4, -1, -1], [-1] * 3, [5, 6, -1], [7, -1, -1], [8, 99, -1]], np.int32)
    free = np.array([1, 2, 50], np.int32)                    # 50 lies outside the pool
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(pkv, tables, lens, new, free, 3, 8, 10, status=status)
    _same(got, R.plan(tables, lens, new, free, 3, 8, 10))
    assert (got[3][2:5] == -1).all()
    assert int(status.item()) == _lib.PA_DEV_BAD_CONTEXT_LEN | _lib.PA_DEV_BAD_BLOCK_ID


def test_plan_equals_host_block_manager(pkv):
    """The same slots, tables and free stack as pa_bm_append_slots gives, step after step."""
    B, blocks, width = 9, 64, 6
    bm = pkv.BlockManager(blocks)
    lens = np.array([1, 15, 16, 17, 31, 32, 5, 48, 2], np.int32)
    for b in range(B):
        bm.alloc_seq(b, int(lens[b]))
    tables, _ = bm.fill_tables(range(B), width)
    used = set(tables[tables >= 0].tolist())
    free = np.array(sorted(set(range(blocks)) - used, reverse=True), np.int32)   # a stack that hands out the lowest
    nf = free.size
    for _ in range(20):
        t, lens2, start, slots, pos, nf2 = _run(pkv, tables, lens, np.ones(B, np.int32), free, nf, B, blocks)
        want, cow = bm.append_slots(range(B))
        assert cow.shape[0] == 0 and np.array_equal(slots, want) and np.array_equal(pos, lens)
        assert np.array_equal(start, np.arange(B + 1))
        tables, lens, nf = t, lens2, nf2
        host, hlens = bm.fill_tables(range(B), width)
        assert np.array_equal(host, tables) and np.array_equal(hlens, lens) and nf == bm.num_free()


def test_plan_empty_batch_and_no_tokens(pkv):
    z = np.zeros(0, np.int32)
    got = _run(pkv, np.zeros((0, 4), np.int32), z, z, np.array([1], np.int32), 1, 5, 4)
    assert got[2].tolist() == [0] and (got[3] == -1).all() and (got[4] == 0).all() and got[5] == 1
    got = _run(pkv, np.zeros((2, 1), np.int32), np.array([0, 3], np.int32), np.zeros(2, np.int32), z, 0, 0, 4)
    assert got[1].tolist() == [0, 3] and got[2].tolist() == [0, 0, 0] and got[5] == 0


def test_plan_into_given_buffers_on_another_stream_and_in_a_graph(pkv):
    rng = np.random.default_rng(3)
    lens, new, tables, free, blocks = _case(rng, 300, 200, 30, 0.5)
    cap = int(new.sum()) + 9
    d = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    t, l, n, f, nf = d(tables), d(lens), d(new), d(free), d(np.array([free.size], np.int32))
    i32 = dict(dtype=torch.int32, device="cuda")
    out = pkv.StepPlan(torch.empty(300, **i32), torch.empty(301, **i32), torch.empty(cap, dtype=torch.int64, device="cuda"),
                       torch.empty(cap, **i32), torch.empty(1, **i32))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert pkv.plan_step(t, l, n, f, nf, cap, blocks, out=out, stream=s).positions is out.positions
    torch.cuda.synchronize()
    want = R.plan(tables, lens, new, free, free.size, cap, blocks)
    take = lambda: [x.cpu().numpy() for x in (t, *out[:4])] + [int(out.num_free.item())]  # noqa: E731
    _same(take(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.plan_step(t, l, n, f, nf, cap, blocks, out=out)
    for x in out:
        x.fill_(77)
    t.copy_(d(tables))
    g.replay()
    torch.cuda.synchronize()
    _same(take(), want)
