"""pa_rotary_turns against 90-digit decimal arithmetic: every frequency is the nearest 64-bit fraction of a
turn, so that far positions keep their angles.  CPU only but for the last test."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import paged_kv_cache_100_gb300 as pkv
from paged_kv_cache_100_gb300.build import build
from tests import block8_ref as R

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")


@pytest.fixture(scope="module", autouse=True)
def _build():
    build()


def exact_turns(rot, base, kind, factor):
    """Turns per position of every pair, to about 85 digits."""
    getcontext().prec = 90
    log_base = Decimal(base).ln()
    if kind == "ntk" and rot > 2:
        log_base += Decimal(factor).ln() * rot / (rot - 2)
    lo, hi = 0, 1
    if kind == "by_parts":
        at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    turns = []
    for i in range(rot // 2):
        theta = (-log_base * 2 * i / rot).exp()
        if kind == "linear":
            theta /= Decimal(factor)
        if kind == "by_parts":
            r = min(max(Decimal(i - lo) / max(Decimal(hi - lo), Decimal("0.001")), Decimal(0)), Decimal(1))
            theta = theta * (1 - r) + theta / Decimal(factor) * r
        turns.append(theta / (2 * PI))
    return turns


@pytest.mark.parametrize("kind,factor", [("none", 1.0), ("linear", 4.0), ("linear", 0.3), ("ntk", 8.0), ("ntk", 0.5), ("by_parts", 8.0),
                                         ("by_parts", 32.5)])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 10.5, 1e30])
def test_turns_are_the_nearest(base, kind, factor):
    for rot in (2, 4, 6, 64, 122, 128, 256):
        got = pkv.rotary_plan(rot, base, scaling=kind, factor=factor, device="cpu").turns.tolist()
        for g, t in zip(got, exact_turns(rot, base, kind, factor)):
            d = abs(Decimal(g % 2 ** 64) - (t - int(t)) * 2 ** 64)
            assert min(d, 2 ** 64 - d) <= Decimal("0.5000001"), (rot, float(d))


def test_turns_too_fast_are_refused():
    for bad in (dict(base=1.5, scaling="ntk", factor=1e-300), dict(base=1e4, scaling="linear", factor=1e-9),
                dict(base=1e4, scaling="linear", factor=1e-300), dict(base=1e4, scaling="by_parts", factor=1e-300)):
        with pytest.raises(pkv.PagedKVError):
            pkv.rotary_plan(64, device="cpu", **bad)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,factor", [("none", 1.0), ("by_parts", 8.0)])
def test_far_positions_keep_their_angles(kind, factor):
    D, base = 128, 500000.0
    pos = [1, 131071, 2 ** 24 + 1, 2 ** 28 - 3, 2 ** 30 + 12345, 2 ** 31 - 1, -5]
    rope = pkv.rotary_plan(D, base, scaling=kind, factor=factor)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(len(pos), 3, D, generator=g)
    pool = torch.zeros(1, 1, 16, D, device="cuda")
    d = x.cuda()
    out = pkv.rope_cache_write(d[:, :1], d[:, 1:2], d[:, 2:], torch.tensor(pos, dtype=torch.int32, device="cuda"), rope, pool,
                               torch.zeros_like(pool), torch.arange(len(pos), device="cuda"))
    turns = exact_turns(D, base, kind, factor)
    frac = np.array([[float((p * t) % 1) for t in turns] for p in pos])       # of a turn, exact before the rounding to float64
    a = rope.attention_factor
    ref, mass = R.rotate(x.double().numpy(), a * np.cos(2 * np.pi * frac), a * np.sin(2 * np.pi * frac), False)
    # the angle to 2^-24 of half a turn (below 2^-22 radians), sincospi to 2^-22, three roundings of 2^-24
    turn = a * (2.0 ** -22 + 2.0 ** -22 + 3 * 2.0 ** -24) * mass[:, :1]
    err = np.abs(out.double().cpu().numpy() - ref[:, :1])
    assert (err <= turn + 2.0 ** -24 * (np.abs(ref[:, :1]) + turn)).all()
