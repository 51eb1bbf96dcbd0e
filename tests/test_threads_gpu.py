"""Calls from several host threads, each on its own stream: a thread whose first CUDA call is one of the
library's, and calls of different sizes at once, none of which may take away what another one needs."""
import threading

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


def _together(calls, rounds):
    """Runs every call again and again in a new thread of its own; returns what was raised and the last results."""
    errors, results = [], [None] * len(calls)
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    start = threading.Barrier(len(calls))

    def loop(i):
        start.wait()
        try:
            for _ in range(rounds):
                results[i] = calls[i](streams[i])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors, results


def test_a_threads_first_call(pkv):
    """Tensors and outputs are there before: nothing but the call itself binds the thread to the device."""
    g = torch.Generator().manual_seed(2)
    lens = [100, 17]
    tables, blocks = R.tables_for(g, lens)
    codes, ks = R.pools(g, blocks, 2, D)
    rows = torch.randn(blocks, 2, 16, D, generator=g).to(torch.bfloat16).cuda()
    c, s = codes.cuda(), ks.cuda()
    table, length, start = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), torch.arange(3, dtype=torch.int32).cuda()
    q = torch.randn(2, 4, D, generator=g).to(torch.bfloat16).cuda()
    head = torch.ones(2, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    calls = [lambda st, o: pkv.decode(q, rows, rows, table, length, out=o, stream=st, workspace=ws),
             lambda st, o: pkv.decode_fp8(q, c, c, head, head, table, length, out=o, stream=st, workspace=ws),
             lambda st, o: pkv.prefill(q, rows, rows, table, length, start, 1, out=o, stream=st, workspace=ws),
             lambda st, o: pkv.decode_block_fp8(q, c, c, s, s, table, length, out=o, stream=st, workspace=ws),
             lambda st, o: pkv.prefill_block_fp8(q, c, c, s, s, table, length, start, 1, out=o, stream=st, workspace=ws)]
    for call in calls:
        want, got = torch.empty_like(q), torch.empty_like(q)
        call(None, want)
        errors, _ = _together([lambda st: call(st, got)], 1)
        assert not errors and torch.equal(got, want)


def test_decodes_of_different_partitions(pkv):
    g = torch.Generator().manual_seed(1)
    lens = [700, 33, 1]
    tables, blocks = R.tables_for(g, lens, width=1024)
    kc, ks = R.pools(g, blocks, 2, D)
    dev = [t.cuda() for t in (kc, kc, ks, ks, torch.from_numpy(tables), torch.tensor(lens, dtype=torch.int32))]
    q = torch.randn(3, 4, D, generator=g).to(torch.bfloat16).cuda()
    sizes = [512, 16384, 4096, 8192]
    want = [pkv.decode_block_fp8(q, *dev, partition_size=p) for p in sizes]
    head = torch.ones(2, device="cuda")
    flat = [pkv.decode_fp8(q, dev[0], dev[1], head, head, dev[4], dev[5], partition_size=p) for p in sizes]
    torch.cuda.synchronize()
    errors, got = _together([lambda s, p=p: pkv.decode_block_fp8(q, *dev, partition_size=p, stream=s) for p in sizes], 3000)
    assert not errors and all(torch.equal(a, b) for a, b in zip(got, want))
    errors, got = _together([lambda s, p=p: pkv.decode_fp8(q, dev[0], dev[1], head, head, dev[4], dev[5], partition_size=p, stream=s)
                             for p in sizes], 3000)
    assert not errors and all(torch.equal(a, b) for a, b in zip(got, flat))


def test_rotary_writes_of_different_sizes(pkv):
    """Thread blocks of 16 and of 64 tokens, whose tables of angles differ in size."""
    dim, calls, checks = 256, [], []
    for n, hkv in ((12000, 1), (40000, 1), (12000, 4)):
        x = torch.randn(n, 2 * hkv, dim, device="cuda", generator=torch.Generator("cuda").manual_seed(n)).to(torch.bfloat16)
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        slots = torch.arange(n, device="cuda")
        pools = [torch.zeros(-(-n // 16), hkv, 16, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(-(-n // 16), hkv, device="cuda") for _ in range(2)]
        rope = pkv.rotary_plan(dim)

        def call(stream, x=x, pos=pos, slots=slots, pools=pools, scales=scales, rope=rope, hkv=hkv):
            pkv.rope_cache_write(None, x[:, :hkv], x[:, hkv:], pos, rope, pools[0], pools[1], slots,
                                 k_scales=scales[0], v_scales=scales[1], stream=stream)

        call(None)
        checks.append((pools, [p.clone() for p in pools]))
        calls.append(call)
    torch.cuda.synchronize()
    errors, _ = _together(calls, 3000)
    assert not errors
    for pools, want in checks:
        assert all(torch.equal(a, b) for a, b in zip(pools, want))
