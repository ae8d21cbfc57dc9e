"""Rotary positions on the host: the table of frequencies against the formulas in
exact arithmetic, and the call's refusals (pointers are never followed)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

P = 1 << 20


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_pass_gb300 as sv
    from speculative_decoding_verify_pass_gb300 import _build
    _build.build()
    return sv


def table(sv, *args, **kw):
    turns, gain = sv.spec_rope_table(*args, device="cpu", **kw)
    return [int(x) for x in turns.numpy().view(np.uint64)], gain


def near(turns, freq):
    """Turns of 2^-64 per position, to a few fp64 roundings of the frequency."""
    want = freq / (2 * math.pi) * 2.0 ** 64
    return abs(turns - want) <= 16 * 2.0 ** -53 * want + 1


@pytest.mark.parametrize("dim", [2, 6, 24, 64, 128, 1024])
@pytest.mark.parametrize("base", [1e4, 5e5, 2.0])
def test_plain_linear_and_base(sv, dim, base):
    plain, gain = table(sv, dim, base)
    assert len(plain) == dim // 2 and gain == 1.0
    assert all(near(t, base ** (-2 * i / dim)) for i, t in enumerate(plain))
    assert near(plain[0], 1.0)
    slow, gain = table(sv, dim, base, sv.SPEC_ROPE_LINEAR, 8.0)
    assert gain == 1.0 and all(near(t, base ** (-2 * i / dim) / 8) for i, t in enumerate(slow))
    if dim > 2:
        b = base * 8.0 ** (dim / (dim - 2))
        wide, gain = table(sv, dim, base, sv.SPEC_ROPE_BASE, 8.0)
        assert gain == 1.0 and all(near(t, b ** (-2 * i / dim)) for i, t in enumerate(wide))
        assert near(wide[0], 1.0) and near(wide[-1], base ** (-2 * (dim // 2 - 1) / dim) / 8)   # the last pair is slowed by the factor


@pytest.mark.parametrize("factor,low,high,context", [(8.0, 1.0, 4.0, 8192), (32.0, 0.5, 3.0, 100), (1.0, 1.0, 4.0, 8192)])
def test_wavelength_ramp(sv, factor, low, high, context):
    got, gain = table(sv, 128, 5e5, sv.SPEC_ROPE_WAVELENGTH, factor, low, high, context)
    assert gain == 1.0
    kept = slowed = between = 0
    for i, t in enumerate(got):
        f = 5e5 ** (-2 * i / 128)
        waves = context * f / (2 * math.pi)
        if waves <= low:
            slowed += 1
            assert near(t, f / factor)
        elif waves >= high:
            kept += 1
            assert near(t, f)
        else:
            between += 1
            a = (waves - low) / (high - low)
            assert near(t, a * f + (1 - a) * f / factor)
    assert kept and slowed and between


def test_parts_ramp_and_its_gain(sv):
    got, gain = table(sv, 64, 1e4, sv.SPEC_ROPE_PARTS, 16.0, 1.0, 32.0, 4096)
    assert gain == pytest.approx(0.1 * math.log(16) + 1, rel=2 ** -23)
    at = [64 * math.log(4096 / (2 * math.pi * n)) / (2 * math.log(1e4)) for n in (32, 1)]
    lo, hi = math.floor(at[0]), math.ceil(at[1])
    assert 0 < lo < hi < 32
    for i, t in enumerate(got):
        f, a = 1e4 ** (-2 * i / 64), min(1.0, max(0.0, (i - lo) / (hi - lo)))
        assert near(t, a * f / 16 + (1 - a) * f)


@pytest.mark.parametrize("low,high,context", [(1.0, 32.0, 1), (1.0, 32.0, 6), (32.0, 64.0, 128), (32.0, 64.0, 200), (1.0, 32.0, 10 ** 9),
                                              (0.5, 1.0, 40)])
@pytest.mark.parametrize("dim,base", [(64, 1e4), (128, 5e5), (4, 1e4), (64, 1.01)])
def test_parts_ramp_at_its_ends(sv, dim, base, low, high, context):
    """Contexts in which no pair turns `low` times, or all turn `high` times: all slowed (pair 0 too), or all kept."""
    got, _ = table(sv, dim, base, sv.SPEC_ROPE_PARTS, 16.0, low, high, context)
    for i, t in enumerate(got):
        f = base ** (-2 * i / dim)
        turns = context * f / (2 * math.pi)
        if turns <= low * base ** (-2 / dim):           # a whole pair past the ramp's end, as it is rounded outwards
            assert near(t, f / 16)
        elif turns >= high * base ** (2 / dim):
            assert near(t, f)
        else:
            assert f / 16 * (1 - 2.0 ** -40) <= t / 2.0 ** 64 * 2 * math.pi <= f * (1 + 2.0 ** -40)


def test_fixed_point_angle_of_far_positions(sv):
    """position * turns modulo 2^64 is the angle to a rounding of the frequency, whatever the position."""
    turns, _ = table(sv, 128, 5e5)
    for i in (0, 1, 17, 63):
        exact = Fraction(turns[i], 1 << 64)
        for pos in (1, 4095, 10 ** 6, 2 ** 31 - 1, -5, -2 ** 31):
            phase = (pos * turns[i]) % (1 << 64)
            assert Fraction(phase, 1 << 64) == (pos * exact) % 1


@pytest.mark.parametrize("over,word", [
    (dict(dim=0), "rotary_dim"), (dict(dim=7), "rotary_dim"), (dict(dim=1026), "rotary_dim"), (dict(base=1.0), "base"),
    (dict(base=float("inf")), "base"), (dict(base=float("nan")), "base"), (dict(kind=5), "scaling"), (dict(kind=-1), "scaling"),
    (dict(kind=1, factor=0.5), "factor"), (dict(kind=4, factor=float("nan")), "factor"), (dict(kind=2, dim=2), "base"),
    (dict(kind=3, low=0.0), "low"), (dict(kind=3, low=4.0), "low"), (dict(kind=4, high=float("inf")), "low"),
    (dict(kind=4, context=0), "context"), (dict(out=None), "null"), (dict(gain=None), "null")])
def test_table_refusals(sv, over, word):
    lib = sv.library()
    out, gain = (ctypes.c_uint64 * 1024)(), ctypes.c_float(0)
    a = dict(dict(dim=128, base=1e4, kind=0, factor=8.0, low=1.0, high=4.0, context=8192, out=out, gain=ctypes.byref(gain)), **over)
    st = lib.spec_rope_table(a["dim"], a["base"], a["kind"], a["factor"], a["low"], a["high"], a["context"], a["out"], a["gain"])
    assert st == sv.SPEC_ERR_INVALID_ARG and word in lib.spec_last_error().decode()


ROPE = dict(x=P, xs=1024, out=P, os=1024, type=0, rows=3, heads=8, hd=128, rot=128, inter=0, inv=0, gain=1.0, turns=P, start=P,
            len=P, nseq=2, pos=None)


def call(sv, over):
    a = dict(ROPE, **over)
    return sv.library().spec_rope(a["x"], a["xs"], a["out"], a["os"], a["type"], a["rows"], a["heads"], a["hd"], a["rot"], a["inter"],
                                  a["inv"], a["gain"], a["turns"], a["start"], a["len"], a["nseq"], a["pos"], None)


@pytest.mark.parametrize("over,word", [
    (dict(x=None), "null"), (dict(out=None), "null"), (dict(turns=None), "null"), (dict(type=3), "type"), (dict(type=-1), "type"),
    (dict(rows=-1), "rows"), (dict(heads=0), "heads"), (dict(heads=4097), "heads"), (dict(hd=12), "head_dim"), (dict(hd=0), "head_dim"),
    (dict(hd=1032), "head_dim"), (dict(rot=130), "rotary_dim"), (dict(rot=0), "rotary_dim"), (dict(rot=9), "rotary_dim"),
    (dict(gain=float("nan")), "gain"), (dict(gain=float("inf")), "gain"), (dict(xs=1016), "strides"), (dict(os=1028), "strides"),
    (dict(xs=1 << 38), "strides"), (dict(type=2, xs=1026), "strides"), (dict(nseq=1025), "nseq"), (dict(nseq=-1), "nseq"),
    (dict(pos=P), "one of the two"), (dict(start=None, len=None), "one of the two"), (dict(len=None), "one of the two"),
    (dict(start=None), "one of the two"), (dict(x=P + 8), "aligned"), (dict(out=P + 4), "aligned"), (dict(turns=P + 4), "aligned"),
    (dict(start=P + 2), "aligned"), (dict(len=P + 1), "aligned"), (dict(start=None, len=None, pos=P + 1), "aligned"),
    (dict(os=2048), "in place")])
def test_rope_refusals(sv, over, word):
    assert call(sv, over) == sv.SPEC_ERR_INVALID_ARG
    assert word in sv.library().spec_last_error().decode()


def test_nothing_to_turn_is_no_error(sv):
    assert call(sv, dict(rows=0, x=None, out=None, turns=None, start=None, len=None)) == 0
    assert call(sv, dict(nseq=0, x=None, out=None)) == 0


def test_a_batch_of_no_sequences_is_no_error(sv):
    """Lengths of no sequences may be a null pointer, which is what an empty tensor has."""
    assert call(sv, dict(nseq=0, len=None)) == 0
    for over in (dict(nseq=0, start=None), dict(nseq=0, start=None, len=None), dict(nseq=0, len=None, pos=P)):
        assert call(sv, over) == sv.SPEC_ERR_INVALID_ARG and "one of the two" in sv.library().spec_last_error().decode()


def test_binding_refuses_host_tensors(sv):
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    for args in ((x, i.long(), i, i), (None, i.long(), i, i), (x[0], i.long(), i, i)):
        with pytest.raises(sv.SpecError) as e:
            sv.spec_rope(*args)
        assert e.value.status == sv.SPEC_ERR_INVALID_ARG
