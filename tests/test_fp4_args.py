"""Refusals of the operators on pools held in 4 bits: CPU only, every check below returns before any
CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_100_gb300 as pkv
from paged_kv_cache_100_gb300 import _lib
from paged_kv_cache_100_gb300.build import build
from tests import fp4_ref as F

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


WRITE = dict(query_out=A, query=2 * A, key=3 * A, value=4 * A, positions=5 * A, turns=6 * A, factor=1.0, rotary_dim=128,
             interleaved=0, key_cache=7 * A, value_cache=8 * A, slots=11 * A, tokens=2, hq=8, hkv=2, dim=128, qo_stride=1024,
             q_stride=1024, k_stride=256, v_stride=256, block_size=16, num_blocks=10, dtype=1, status=None, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(tokens=-1), BAD), (dict(hq=-1), BAD), (dict(hkv=0), BAD), (dict(dim=0), BAD), (dict(rotary_dim=127), BAD),
    (dict(rotary_dim=130), BAD), (dict(rotary_dim=-2), BAD), (dict(block_size=8), BAD), (dict(num_blocks=0), BAD),
    (dict(factor=float("nan")), BAD), (dict(factor=0.0), BAD), (dict(dtype=2), BAD), (dict(query=None), BAD),
    (dict(query_out=None), BAD), (dict(key=None), BAD), (dict(value=None), BAD), (dict(positions=None), BAD),
    (dict(turns=None), BAD), (dict(slots=None), BAD), (dict(key_cache=None), BAD), (dict(value_cache=8 * A + 8), BAD),
    (dict(query=2 * A + 8), BAD), (dict(key=3 * A + 2), BAD), (dict(q_stride=1023), BAD), (dict(k_stride=128), BAD),
    (dict(v_stride=260), BAD), (dict(slots=11 * A + 4), BAD), (dict(turns=6 * A + 4), BAD), (dict(positions=5 * A + 2), BAD),
    (dict(query_out=2 * A + 2048), BAD), (dict(query_out=3 * A), BAD), (dict(query_out=2 * A, qo_stride=2048), BAD),
    (dict(dim=272, rotary_dim=0, q_stride=1 << 14, qo_stride=1 << 14, k_stride=1 << 12, v_stride=1 << 12), UNSUPPORTED),
    (dict(dim=100, rotary_dim=0), UNSUPPORTED), (dict(dim=24, rotary_dim=0), UNSUPPORTED),
    (dict(tokens=0, query=None, key=None), OK)])
def test_write_refuses(lib, over, expect):
    assert _call(lib.pa_rope_cache_write_fp4, WRITE, over) == expect


READ = dict(key_out=A, value_out=2 * A, key_cache=3 * A, value_cache=4 * A, tables=5 * A, lens=6 * A, num_seqs=2, hkv=2,
            dim=128, block_size=16, max_blocks=4, num_blocks=10, longest=0, window=0, dtype=1, status=None, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(num_seqs=-1), BAD), (dict(hkv=0), BAD), (dict(dim=-16), BAD), (dict(block_size=32), BAD), (dict(max_blocks=-1), BAD),
    (dict(max_blocks=1 << 28), BAD), (dict(num_blocks=0), BAD), (dict(longest=-1), BAD), (dict(window=-1), BAD),
    (dict(dtype=2), BAD), (dict(key_out=None), BAD), (dict(value_out=None), BAD), (dict(key_cache=None), BAD),
    (dict(tables=None), BAD), (dict(lens=None), BAD), (dict(key_out=A + 8), BAD), (dict(value_cache=4 * A + 1), BAD),
    (dict(tables=5 * A + 2), BAD), (dict(dim=40), UNSUPPORTED), (dict(dim=512), UNSUPPORTED),
    (dict(hkv=1 << 22), UNSUPPORTED), (dict(num_seqs=1 << 20, max_blocks=1 << 12), UNSUPPORTED),
    (dict(key_out=2 * A), BAD), (dict(key_out=2 * A + 65520), BAD), (dict(key_out=2 * A - 65520), BAD),
    (dict(value_out=3 * A + 16), BAD), (dict(key_out=4 * A - 65520), BAD), (dict(key_out=5 * A - 65520), BAD),
    (dict(value_out=6 * A - 65520), BAD), (dict(num_seqs=0, key_out=None), OK), (dict(max_blocks=0, tables=None), OK)])
def test_read_refuses(lib, over, expect):
    assert _call(lib.pa_cache_read_fp4, READ, over) == expect


DECODE = dict(out=A, query=2 * A, key_cache=3 * A, value_cache=4 * A, tables=7 * A, lens=8 * A, start=None, num_seqs=1,
              tokens=1, hq=8, hkv=2, dim=128, block_size=16, max_blocks=4, num_blocks=8, scale=0.1, window=0, partition=0,
              workspace=None, workspace_bytes=0, status=None, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(num_seqs=-1), BAD), (dict(tokens=2), BAD), (dict(tokens=-1), BAD), (dict(hq=7), BAD), (dict(hkv=0), BAD),
    (dict(block_size=8), BAD), (dict(max_blocks=-1), BAD), (dict(num_blocks=0), BAD), (dict(scale=float("nan")), BAD),
    (dict(window=-1), BAD), (dict(partition=24), BAD), (dict(partition=32768), BAD), (dict(out=None), BAD),
    (dict(query=None), BAD), (dict(tables=None), BAD), (dict(lens=None), BAD), (dict(out=A + 8), BAD),
    (dict(key_cache=3 * A + 4), BAD), (dict(start=9 * A + 2), BAD), (dict(dim=96), UNSUPPORTED),
    (dict(max_blocks=1000), WORKSPACE), (dict(max_blocks=1000, workspace=A, workspace_bytes=100), WORKSPACE),
    (dict(num_seqs=1 << 20, tokens=1 << 20, hq=1 << 12, hkv=1 << 12), UNSUPPORTED),
    (dict(num_seqs=0, tokens=0, out=None, query=None), OK), (dict(start=9 * A, tokens=0, query=None), OK)])
def test_decode_refuses(lib, over, expect):
    assert _call(lib.pa_decode_fp4, DECODE, over) == expect


def test_decode_workspace(lib):
    f, bad = lib.pa_decode_fp4_workspace_bytes, ctypes.c_size_t(-1).value
    assert f(4, 8, 2, 128, 4, 16, 0, 0) == 0
    assert f(4, 8, 2, 64, 64, 16, 0, 512) >= 4 * 8 * 2 * (64 * 4 + 8)
    assert f(4, 8, 2, 128, 64, 16, 30, 512) == 0              # a window inside one partition
    for args in ((-1, 8, 2, 128, 4, 16, 0, 0), (4, 7, 2, 128, 4, 16, 0, 0), (4, 8, 2, 32, 4, 16, 0, 0),
                 (4, 8, 2, 128, 4, 8, 0, 0), (4, 8, 2, 128, 4, 16, -1, 0), (4, 8, 2, 128, 4, 16, 0, 17)):
        assert f(*args) == bad


PREFILL = dict(out=A, query=2 * A, key_cache=3 * A, value_cache=4 * A, tables=7 * A, lens=8 * A, start=9 * A, num_seqs=1, hq=8,
               hkv=2, dim=128, block_size=16, max_blocks=4, num_blocks=8, tokens=4, longest_chunk=4, longest=0, scale=0.1,
               window=0, workspace=10 * A, workspace_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("over,expect", [
    (dict(num_seqs=-1), BAD), (dict(hq=7), BAD), (dict(tokens=-1), BAD), (dict(longest_chunk=-1), BAD), (dict(longest=-1), BAD),
    (dict(window=-1), BAD), (dict(scale=float("nan")), BAD), (dict(block_size=8), BAD), (dict(num_blocks=0), BAD),
    (dict(max_blocks=0), BAD), (dict(max_blocks=1 << 28), BAD), (dict(out=None), BAD), (dict(start=None), BAD),
    (dict(tables=None), BAD), (dict(lens=8 * A + 1), BAD), (dict(query=2 * A + 8), BAD), (dict(dim=64), UNSUPPORTED),
    (dict(hq=6), UNSUPPORTED), (dict(hq=64), UNSUPPORTED), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=500), WORKSPACE), (dict(workspace=10 * A + 4), WORKSPACE),
    (dict(num_seqs=1 << 16, max_blocks=1 << 12), UNSUPPORTED), (dict(num_seqs=0, out=None), OK), (dict(tokens=0, out=None), OK),
    (dict(longest_chunk=0, out=None), OK)])
def test_prefill_refuses(lib, over, expect):
    assert _call(lib.pa_prefill_fp4, PREFILL, over) == expect


def test_prefill_workspace(lib):
    f, bad = lib.pa_prefill_fp4_workspace_bytes, ctypes.c_size_t(-1).value
    block = 2 * 2 * 16 * 128 * 2                                     # keys and values of two heads, staged
    long = (4000, 4000)                                              # rows, and of the longest chunk: staged
    assert f(3, 8, 2, 128, 10, *long, 0, 0) >= 30 * block and f(3, 8, 2, 128, 10, *long, 33, 0) < 10 * block
    assert f(3, 8, 2, 128, 10, *long, 33, 0) >= 9 * block and f(3, 8, 2, 128, 10, *long, 1000, 0) == f(3, 8, 2, 128, 10, *long, 0, 0)
    assert f(1 << 20, 8, 8, 128, 1 << 10, 1 << 20, 100, 0, 0) > 1 << 45      # counted in 64 bits
    assert f(1, 8, 2, 128, 512, 1, 1, 0, 0) < 512 * block            # a few rows: as a decode
    for args in ((-1, 8, 2, 128, 10, 1, 1, 0, 0), (3, 7, 2, 128, 10, 1, 1, 0, 0), (3, 8, 0, 128, 10, 1, 1, 0, 0),
                 (3, 8, 2, 64, 10, 1, 1, 0, 0), (3, 8, 2, 128, -1, 1, 1, 0, 0), (3, 8, 2, 128, 10, -1, 1, 0, 0),
                 (3, 8, 2, 128, 10, 1, -1, 0, 0), (3, 8, 2, 128, 10, 1, 1, -1, 0), (3, 8, 2, 128, 10, 1, 1, 0, -1)):
        assert f(*args) == bad
    assert pkv.prefill_fp4_workspace_bytes(3, 8, 2, 128, 10, *long, 33) == f(3, 8, 2, 128, 10, *long, 33, 0)
    assert pkv.decode_fp4_workspace_bytes(4, 8, 2, 128, 64, 512) == lib.pa_decode_fp4_workspace_bytes(4, 8, 2, 128, 64, 16, 0, 512)
    with pytest.raises(ValueError):
        pkv.prefill_fp4_workspace_bytes(3, 8, 2, 128, -1, 1, 1)
    with pytest.raises(ValueError):
        pkv.decode_fp4_workspace_bytes(3, 2, 2, 96, 1)


def _z(*s, dt=torch.int32):
    return torch.zeros(*s, dtype=dt)


def test_bindings_refuse_cpu_tensors_shapes_and_types():
    bf, i64 = torch.bfloat16, torch.int64
    pool, q = pkv.fp4_pool(2, 1, 128, device="cpu"), _z(1, 1, 128, dt=bf)
    assert pool.shape == (2, 1, 16, 72) and pool.dtype == torch.uint8
    for bad in (0, 24, 272, -16):
        with pytest.raises(ValueError):
            pkv.fp4_pool(2, 1, bad, device="cpu")
    calls = (lambda q=q, kc=pool, vc=pool, **o: pkv.rope_cache_write_fp4(q, q, q, None, None, kc, vc, _z(1, dt=i64), **o),
             lambda q=q, kc=pool, vc=pool, **o: pkv.cache_read_fp4(kc, vc, _z(1, 1), _z(1), **o),
             lambda q=q, kc=pool, vc=pool, **o: pkv.decode_fp4(q, kc, vc, _z(1, 1), _z(1), **o),
             lambda q=q, kc=pool, vc=pool, **o: pkv.prefill_fp4(q, kc, vc, _z(1, 1), _z(1), _z(2), 1, **o))
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="CUDA"):
            call()
        with pytest.raises(TypeError, match="uint8"):
            call(kc=pool.to(torch.int8))
        with pytest.raises(ValueError, match="4-bit pools"):
            call(kc=_z(2, 1, 16, 64, dt=torch.uint8), vc=_z(2, 1, 16, 64, dt=torch.uint8))
        with pytest.raises(ValueError, match="4-bit pools"):
            call(vc=pkv.fp4_pool(3, 1, 128, device="cpu"))
        if i != 1:
            with pytest.raises(TypeError):
                call(q=q.half())
            with pytest.raises(ValueError):
                call(q=_z(1, 1, 64, dt=bf))
    with pytest.raises(TypeError, match="bfloat16"):
        pkv.decode_fp4(q.float(), pool, pool, _z(1, 1), _z(1))
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        pkv.cache_read_fp4(pool, pool, _z(1, 1), _z(1), dtype=torch.float16)
    for width in (0, -3):
        with pytest.raises(ValueError, match="max_context_len"):
            pkv.cache_read_fp4(pool, pool, _z(1, 1), _z(1), max_context_len=width)
        with pytest.raises(ValueError, match="max_context_len"):
            pkv.prefill_fp4(q, pool, pool, _z(1, 1), _z(1), _z(2), 1, max_context_len=width)
    with pytest.raises(ValueError, match="block_tables"):
        pkv.cache_read_fp4(pool, pool, _z(2, 1), _z(1))
    with pytest.raises(ValueError, match="context_lens"):
        pkv.decode_fp4(q, pool, pool, _z(2, 1), _z(2))
    for start in (_z(2), _z(4), _z(3, 1)):
        with pytest.raises(ValueError, match="query_start"):
            pkv.decode_fp4(q, pool, pool, _z(2, 1), _z(2), query_start=start)
        with pytest.raises(ValueError, match="query_start"):
            pkv.prefill_fp4(q, pool, pool, _z(2, 1), _z(2), start, 1)


def test_the_reference_itself():
    """The plain encoding: every code and scale is its own nearest one, and errors are within half a step."""
    assert F.SCALES[-1] == 10240 and F.SCALES[1] == 2.0 ** -17
    half = (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(F.scales_of(np.arange(0xF8)), half[:0xF8])
    rng = np.random.default_rng(0)
    for byte in (1, 7, 8, 100, 0xE2):
        c = rng.choice(np.concatenate([F.CODES, -F.CODES]), (50, 16))
        c[:, 0] = 6
        code, b = F.encode(c * F.SCALES[byte])
        assert (b == byte).all() and np.array_equal(code, c)
    x = rng.standard_normal((1000, 64)) * 2.0 ** rng.integers(-12, 12, (1000, 1))
    code, byte = F.encode(x)
    s = np.repeat(F.SCALES[byte], 16, -1)
    # a scale is off by at most 2^-4 of itself, so the largest element's code is 6 and off by as much or half a step
    assert (np.abs(F.values_of(code, byte) - x) <= s * np.where(np.abs(x) < 4 * s, 0.5, 1.0) + 1e-12).all()
    pool = F.pack(code.reshape(125, 8, 64)[:120].reshape(30, 2, 16, 64), byte.reshape(125, 8, 4)[:120].reshape(30, 2, 16, 4))
    assert np.array_equal(F.unpack(pool)[2], F.values_of(code, byte).reshape(125, 8, 64)[:120].reshape(30, 2, 16, 64))
