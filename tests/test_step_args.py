"""Refusals of the step operators (plan, rotary write, block-scaled attention): CPU only, every
check below returns before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_100_gb300 as pkv
from paged_kv_cache_100_gb300 import _lib
from paged_kv_cache_100_gb300.build import build
from tests import block8_ref as R

OK, BAD, UNSUPPORTED, WORKSPACE = _lib.PA_OK, _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED, _lib.PA_ERR_WORKSPACE
A = 1 << 20     # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.lib()


def _call(fn, defaults, over):
    a = dict(defaults)
    assert set(over) <= set(a)
    a.update(over)
    return fn(*a.values())


PLAN = dict(block_tables=A, context_lens=2 * A, new_lens=3 * A, free_blocks=4 * A, num_free=5 * A, lens_out=6 * A,
            query_start=7 * A, slots=8 * A, positions=9 * A, free_out=10 * A, num_seqs=4, max_blocks=8, block_size=16,
            num_blocks=100, free_capacity=10, token_capacity=64, status=None, stream=None)


@pytest.mark.parametrize("over", [
    dict(num_seqs=-1), dict(max_blocks=-1), dict(block_size=32), dict(num_blocks=0), dict(free_capacity=-1),
    dict(token_capacity=-1), dict(max_blocks=1 << 28), dict(context_lens=None), dict(new_lens=None), dict(query_start=None),
    dict(num_free=None), dict(free_out=None), dict(slots=None), dict(positions=None), dict(block_tables=None),
    dict(free_blocks=None), dict(slots=8 * A + 4), dict(positions=9 * A + 2), dict(context_lens=2 * A + 1),
    dict(lens_out=2 * A), dict(lens_out=2 * A + 12), dict(free_out=5 * A), dict(query_start=3 * A - 16),
    dict(positions=8 * A + 8 * 63), dict(block_tables=4 * A + 36)])
def test_plan_refuses(lib, over):
    assert _call(lib.pa_plan_step, PLAN, over) == BAD


def test_plan_refuses_a_capacity_past_its_indexes(lib):
    assert _call(lib.pa_plan_step, PLAN, dict(token_capacity=(1 << 30) + 1, positions=1 << 40, free_out=1 << 44)) == UNSUPPORTED


ROPE = dict(query_out=A, query=2 * A, key=3 * A, value=4 * A, positions=5 * A, turns=6 * A, factor=1.0, rotary_dim=128,
            interleaved=0, key_cache=7 * A, value_cache=8 * A, k_scales=9 * A, v_scales=10 * A, slots=11 * A, tokens=2,
            hq=8, hkv=2, dim=128, qo_stride=1024, q_stride=1024, k_stride=256, v_stride=256, block_size=16,
            num_blocks=10, dtype=1, cache_dtype=2, status=None, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(tokens=-1), BAD), (dict(hq=-1), BAD), (dict(hkv=0), BAD), (dict(dim=0), BAD), (dict(rotary_dim=127), BAD),
    (dict(rotary_dim=130), BAD), (dict(rotary_dim=-2), BAD), (dict(block_size=8), BAD), (dict(num_blocks=0), BAD),
    (dict(factor=float("nan")), BAD), (dict(factor=float("inf")), BAD), (dict(dtype=2), BAD), (dict(cache_dtype=0), BAD),
    (dict(query=None), BAD), (dict(query_out=None), BAD), (dict(key=None), BAD), (dict(value=None), BAD),
    (dict(positions=None), BAD), (dict(turns=None), BAD), (dict(slots=None), BAD), (dict(key_cache=None), BAD),
    (dict(k_scales=None), BAD), (dict(v_scales=10 * A + 2), BAD), (dict(query=2 * A + 8), BAD), (dict(key=3 * A + 2), BAD),
    (dict(q_stride=1023), BAD), (dict(q_stride=1025), BAD), (dict(k_stride=128), BAD), (dict(v_stride=260), BAD),
    (dict(qo_stride=1000), BAD), (dict(query=A, q_stride=2048), BAD), (dict(slots=11 * A + 4), BAD),
    (dict(turns=6 * A + 4), BAD), (dict(dim=264, rotary_dim=0, q_stride=1 << 14, qo_stride=1 << 14, k_stride=1 << 12,
                                        v_stride=1 << 12), UNSUPPORTED),
    (dict(dim=100, rotary_dim=0), UNSUPPORTED), (dict(dim=24, rotary_dim=0), UNSUPPORTED),
    (dict(tokens=0, query=None, key=None), OK)])
def test_rope_write_refuses(lib, over, expect):
    assert _call(lib.pa_rope_cache_write, ROPE, over) == expect


@pytest.mark.parametrize("over", [
    dict(query_out=2 * A + 2048), dict(query_out=2 * A - 2048), dict(query_out=2 * A + 16, q_stride=2048, qo_stride=2048),
    dict(query_out=2 * A, qo_stride=2048), dict(query_out=3 * A), dict(query_out=4 * A + 512, v_stride=1024),
    dict(query=2 * A, query_out=2 * A, key=2 * A + 2032, q_stride=1536, qo_stride=1536, k_stride=1536)])
def test_rope_write_refuses_outputs_over_inputs(lib, over):
    assert _call(lib.pa_rope_cache_write, ROPE, over) == BAD


DECODE = dict(out=A, query=2 * A, key_cache=3 * A, value_cache=4 * A, k_scales=5 * A, v_scales=6 * A, tables=7 * A,
              lens=8 * A, num_seqs=1, hq=8, hkv=2, dim=128, block_size=16, max_blocks=4, num_blocks=8, scale=0.1, window=0,
              partition=0, workspace=None, workspace_bytes=0, status=None, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(num_seqs=-1), BAD), (dict(hq=7), BAD), (dict(hkv=0), BAD), (dict(block_size=8), BAD), (dict(max_blocks=-1), BAD),
    (dict(num_blocks=0), BAD), (dict(scale=float("nan")), BAD), (dict(window=-1), BAD), (dict(partition=24), BAD),
    (dict(partition=32768), BAD), (dict(out=None), BAD), (dict(query=None), BAD), (dict(k_scales=None), BAD),
    (dict(v_scales=None), BAD), (dict(tables=None), BAD), (dict(lens=None), BAD), (dict(out=A + 8), BAD),
    (dict(key_cache=3 * A + 4), BAD), (dict(k_scales=5 * A + 2), BAD), (dict(dim=64), UNSUPPORTED),
    (dict(num_blocks=1 << 26), UNSUPPORTED), (dict(max_blocks=1000), WORKSPACE),
    (dict(max_blocks=1000, workspace=A, workspace_bytes=100), WORKSPACE), (dict(num_seqs=0, out=None, query=None), OK)])
def test_decode_block_fp8_refuses(lib, over, expect):
    assert _call(lib.pa_decode_block_fp8, DECODE, over) == expect


def test_decode_block_fp8_workspace(lib):
    f, bad = lib.pa_decode_block_fp8_workspace_bytes, ctypes.c_size_t(-1).value
    assert f(4, 8, 2, 128, 4, 16, 0, 0) == 0
    assert f(4, 8, 2, 128, 64, 16, 0, 512) >= 4 * 8 * 2 * (128 * 4 + 8)
    assert f(4, 8, 2, 128, 64, 16, 30, 512) == 0              # a window inside one partition
    for args in ((-1, 8, 2, 128, 4, 16, 0, 0), (4, 7, 2, 128, 4, 16, 0, 0), (4, 8, 2, 64, 4, 16, 0, 0),
                 (4, 8, 2, 128, 4, 8, 0, 0), (4, 8, 2, 128, 4, 16, -1, 0), (4, 8, 2, 128, 4, 16, 0, 17)):
        assert f(*args) == bad


PREFILL = dict(out=A, query=2 * A, key_cache=3 * A, value_cache=4 * A, k_scales=5 * A, v_scales=6 * A, tables=7 * A,
               lens=8 * A, start=9 * A, num_seqs=1, hq=8, hkv=2, dim=128, block_size=16, max_blocks=4, num_blocks=8,
               tokens=5, longest=5, scale=0.1, window=0, workspace=10 * A, workspace_bytes=1 << 20, status=None, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(num_seqs=-1), BAD), (dict(hq=7), BAD), (dict(block_size=8), BAD), (dict(max_blocks=-1), BAD),
    (dict(num_blocks=0), BAD), (dict(tokens=-1), BAD), (dict(longest=-1), BAD), (dict(window=-1), BAD),
    (dict(scale=float("nan")), BAD), (dict(out=None), BAD), (dict(start=None), BAD), (dict(k_scales=None), BAD),
    (dict(v_scales=6 * A + 1), BAD), (dict(query=2 * A + 8), BAD), (dict(tables=None), BAD), (dict(dim=64), UNSUPPORTED),
    (dict(hq=6), UNSUPPORTED), (dict(hq=64), UNSUPPORTED), (dict(num_blocks=1 << 26), UNSUPPORTED),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=16), WORKSPACE), (dict(workspace=10 * A + 8), WORKSPACE),
    (dict(max_blocks=512, workspace_bytes=4096), WORKSPACE),          # cut along the context: partial outputs
    (dict(num_seqs=0, out=None), OK), (dict(tokens=0, out=None), OK), (dict(longest=0, out=None), OK)])
def test_prefill_block_fp8_refuses(lib, over, expect):
    assert _call(lib.pa_prefill_block_fp8, PREFILL, over) == expect


def test_prefill_block_fp8_workspace(lib):
    f, bad = lib.pa_prefill_block_fp8_workspace_bytes, ctypes.c_size_t(-1).value
    assert f(16, 64, 8, 128, 544, 8192, 512, 0) < 4096        # enough items: the ticket alone
    assert f(1, 64, 8, 128, 513, 16, 16, 0) >= 16 * 64 * 2 * (128 * 4 + 8)
    assert f(1, 64, 8, 128, 513, 16, 16, 100) < 4096          # a short window is not cut
    for args in ((-1, 8, 2, 128, 4, 5, 5, 0), (1, 7, 2, 128, 4, 5, 5, 0), (1, 8, 2, 64, 4, 5, 5, 0),
                 (1, 6, 2, 128, 4, 5, 5, 0), (1, 8, 2, 128, -4, 5, 5, 0), (1, 8, 2, 128, 4, 5, 5, -1)):
        assert f(*args) == bad


def test_rotary_turns(lib):
    for kind, factor in (("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("by_parts", 8.0)):
        for rot in (2, 6, 64, 122, 128):
            p = pkv.rotary_plan(rot, 500000.0, scaling=kind, factor=factor, device="cpu")
            t = np.array([int(x) % (1 << 64) for x in p.turns.tolist()], dtype=np.float64) * 2.0 ** -64
            cos, sin = R.rotary_angles(np.ones(1), rot, 500000.0, kind, factor)
            a = float(np.hypot(cos[0, 0], sin[0, 0]))
            assert abs(p.attention_factor - a) < 1e-6
            assert np.allclose(a * np.cos(2 * np.pi * t), cos[0], atol=1e-14)
            assert np.allclose(a * np.sin(2 * np.pi * t), sin[0], atol=1e-14)
    assert pkv.rotary_plan(0, device="cpu").turns.numel() == 0
    for bad in (dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, factor=0.0),
                dict(rotary_dim=8, base=float("inf")), dict(rotary_dim=8, scaling="by_parts", original_context=0),
                dict(rotary_dim=8, scaling="by_parts", beta_fast=-1.0)):
        with pytest.raises(pkv.PagedKVError):
            pkv.rotary_plan(device="cpu", **bad)
    with pytest.raises(ValueError):
        pkv.rotary_plan(8, scaling="other", device="cpu")


def test_bindings_refuse_cpu_tensors():
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)  # noqa: E731
    kc, sc = z(2, 1, 16, 128, dt=torch.uint8), z(2, 1, dt=torch.float32)
    q = z(1, 1, 128, dt=torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.plan_step(z(1, 1), z(1), z(1), z(1), z(1), 1, 4)
    with pytest.raises(ValueError):
        pkv.rope_cache_write(q, q, q, None, None, kc, kc, z(1, dt=torch.int64), k_scales=sc, v_scales=sc)
    with pytest.raises(ValueError):
        pkv.decode_block_fp8(q, kc, kc, sc, sc, z(1, 1), z(1))


def test_bindings_refuse_shapes_and_types():
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)  # noqa: E731
    kc, sc = z(2, 1, 16, 128, dt=torch.uint8), z(2, 1, dt=torch.float32)
    q = z(1, 1, 128, dt=torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.plan_step(z(2, 1), z(1), z(2), z(1), z(1), 1, 4)
    with pytest.raises(ValueError):
        pkv.decode_block_fp8(q, kc, kc, sc[:1], sc, z(1, 1), z(1))
    with pytest.raises(TypeError):
        pkv.decode_block_fp8(q.float(), kc, kc, sc, sc, z(1, 1), z(1))
    with pytest.raises(ValueError):
        pkv.decode_block_fp8(q, kc, kc, sc, sc, z(1, 1), z(2))
    with pytest.raises(ValueError):
        pkv.decode_block_fp8(q, z(2, 1, 8, 128, dt=torch.uint8), kc, sc, sc, z(1, 1), z(1))


DECODE_ROWS = dict(out=A, query=2 * A, key_cache=3 * A, value_cache=4 * A, k_scales=5 * A, v_scales=6 * A, tables=7 * A,
                   lens=8 * A, start=9 * A, num_seqs=3, tokens=2, hq=8, hkv=2, dim=128, block_size=16, max_blocks=4, num_blocks=8,
                   scale=0.1, window=0, partition=0, workspace=None, workspace_bytes=0, status=None, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(tokens=-1), BAD), (dict(start=None), BAD), (dict(start=9 * A + 2), BAD), (dict(num_seqs=-1), BAD), (dict(hq=7), BAD),
    (dict(query=None), BAD), (dict(dim=64), UNSUPPORTED), (dict(max_blocks=4000), WORKSPACE),
    (dict(tokens=0, query=None), OK), (dict(num_seqs=0, tokens=0, start=None), OK), (dict(num_seqs=0), OK)])
def test_decode_block_fp8_rows_refuses(lib, over, expect):
    assert _call(lib.pa_decode_block_fp8_rows, DECODE_ROWS, over) == expect


def test_decode_binding_checks_query_start():
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)  # noqa: E731
    kc, sc = z(2, 1, 16, 128, dt=torch.uint8), z(2, 1, dt=torch.float32)
    q = z(1, 1, 128, dt=torch.bfloat16)
    for start in (z(2), z(4), z(3, 1)):
        with pytest.raises(ValueError, match="query_start"):
            pkv.decode_block_fp8(q, kc, kc, sc, sc, z(2, 1), z(2), query_start=start)
    with pytest.raises(TypeError, match="query_start"):
        pkv.decode_block_fp8(q, kc, kc, sc, sc, z(2, 1), z(2), query_start=3)


def test_block_scales_refusals(lib):
    copy = dict(kc=A, vc=2 * A, ks=3 * A, vs=4 * A, pairs=5 * A, n=1, hkv=2, dim=128, block=16, blocks=4, status=None, stream=None)
    for over, expect in ((dict(ks=None), BAD), (dict(vs=None), BAD), (dict(ks=3 * A + 2), BAD), (dict(kc=None), BAD), (dict(pairs=None), BAD),
                         (dict(blocks=0), BAD), (dict(block=8), BAD), (dict(n=-1), BAD), (dict(n=0, ks=None), OK)):
        assert _call(lib.pa_block_copy_scaled, copy, over) == expect
    swap = dict(kc=A, vc=2 * A, ks=3 * A, vs=4 * A, ids=5 * A, n=1, staging=6 * A, scales=7 * A, hkv=2, dim=128, block=16, blocks=4,
                status=None, stream=None)
    for fn in (lib.pa_swap_out_scaled, lib.pa_swap_in_scaled):
        for over, expect in ((dict(ks=None), BAD), (dict(vs=None), BAD), (dict(scales=None), BAD), (dict(scales=7 * A + 1), BAD),
                             (dict(staging=None), BAD), (dict(ids=None), BAD), (dict(n=-1), BAD), (dict(n=0, ks=None, scales=None), OK)):
            assert _call(fn, swap, over) == expect
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)  # noqa: E731
    codes, rows, sc = z(2, 1, 16, 128, dt=torch.uint8), z(2, 1, 16, 128, dt=torch.bfloat16), z(2, 1, dt=torch.float32)
    with pytest.raises(ValueError, match="k_scales"):
        pkv.block_copy(codes, codes, z(1, 2), k_scales=sc)
    with pytest.raises(ValueError, match="k_scales"):
        pkv.block_copy(codes, codes, z(1, 2), k_scales=sc[:1], v_scales=sc)
    with pytest.raises(TypeError, match="E4M3"):
        pkv.block_copy(rows, rows, z(1, 2), k_scales=sc, v_scales=sc)


def test_rope_write_refuses_more_tokens_than_it_counts(lib):
    wide = dict(tokens=(1 << 26) + 1, query_out=1 << 50, query=1 << 51, key=1 << 52, value=1 << 53)
    assert _call(lib.pa_rope_cache_write, ROPE, wide) == UNSUPPORTED
