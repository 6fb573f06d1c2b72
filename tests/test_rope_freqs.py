"""rope_freqs (host only): the fixed-point frequency table against the formulas in
64 bits, its refusals, and the exactness of position * F mod 2^64 in integers."""
import math

import pytest
import torch

import fp8_kv_cache_write_gb300 as fk


@pytest.fixture(scope="module", autouse=True)
def built():
    fk.build()


def _theta(freqs):
    return [int(f) * 2 * math.pi / 2 ** 64 for f in freqs.tolist()]


def _close(got, want):
    # powers and logarithms of the host's libm: a few units in the last place
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert abs(a - b) <= 16 * 2.0 ** -53 * abs(b) + 2 * math.pi * 2.0 ** -64, (a, b)


@pytest.mark.parametrize("rd,base", [(64, 10000.0), (128, 500000.0), (16, 2.0), (2, 10000.0)])
def test_plain_linear_and_ntk(rd, base):
    f, m = fk.rope_freqs(rd, base)
    plain = [base ** (-2 * i / rd) for i in range(rd // 2)]
    assert m == 1.0 and f.dtype == torch.int64
    _close(_theta(f), plain)
    f, m = fk.rope_freqs(rd, base, scaling=fk.ROPE_LINEAR, factor=4.0)
    _close(_theta(f), [t / 4 for t in plain])
    if rd > 2:
        f, m = fk.rope_freqs(rd, base, scaling=fk.ROPE_NTK, factor=3.0)
        b = base * 3.0 ** (rd / (rd - 2))
        _close(_theta(f), [b ** (-2 * i / rd) for i in range(rd // 2)])
        # the lowest frequency is the interpolated one
        assert _theta(f)[-1] == pytest.approx(plain[-1] / 3.0, rel=1e-12)


def test_bands():
    rd, base, factor, ctx = 128, 500000.0, 8.0, 8192
    f, m = fk.rope_freqs(rd, base, scaling=fk.ROPE_BANDS, factor=factor, original_context=ctx,
                         low=1.0, high=4.0)
    want = []
    for i in range(rd // 2):
        t = base ** (-2 * i / rd)
        turns = ctx * t / (2 * math.pi)
        w = min(1.0, max(0.0, (turns - 1.0) / 3.0))
        want.append((1 - w) * t / factor + w * t)
    assert m == 1.0
    _close(_theta(f), want)


def test_yarn():
    rd, base, factor, ctx = 64, 10000.0, 40.0, 4096
    f, m = fk.rope_freqs(rd, base, scaling=fk.ROPE_YARN, factor=factor, original_context=ctx)
    assert m == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-7)
    dim = lambda turns: rd * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = math.floor(dim(32.0)), math.ceil(dim(1.0))
    assert 0 < lo < hi < rd // 2
    want = []
    for i in range(rd // 2):
        t = base ** (-2 * i / rd)
        w = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        want.append(t / factor * w + t * (1 - w))
    _close(_theta(f), want)


def test_the_table_keeps_far_angles():
    # position * F mod 2^64 against exact rational turns of the table itself
    f, _ = fk.rope_freqs(128, 500000.0)
    for p in (1, 131071, (1 << 31) + 7, -5):
        for F in f.tolist()[:5]:
            turns = (p * F) % (1 << 64) / 2 ** 64
            want = (p * (F * 2 * math.pi / 2 ** 64)) / (2 * math.pi) % 1.0
            d = abs(turns - want)
            assert min(d, 1 - d) < abs(p) * 2.0 ** -50


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(base=1.0),
                                dict(base=float("nan")), dict(base=float("inf")), dict(scaling=9),
                                dict(scaling=fk.ROPE_LINEAR, factor=0.5),
                                dict(scaling=fk.ROPE_LINEAR, factor=float("nan")),
                                dict(rotary_dim=2, scaling=fk.ROPE_NTK, factor=2.0),
                                dict(scaling=fk.ROPE_YARN, factor=2.0),
                                dict(scaling=fk.ROPE_BANDS, factor=2.0, original_context=100, low=4.0,
                                     high=4.0),
                                dict(scaling=fk.ROPE_BANDS, factor=2.0, original_context=100, low=0.0)])
def test_refusals(kw):
    args = dict(rotary_dim=64, base=10000.0)
    args.update(kw)
    with pytest.raises(fk.Fp8kvError) as e:
        fk.rope_freqs(**args)
    assert e.value.status == -1
