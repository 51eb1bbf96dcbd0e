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
