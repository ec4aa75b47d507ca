"""Pins of the packed-block oracle (oracle/packed.py): hand-written values,
ties, clamps and the error bounds the format promises.  No GPU."""
import numpy as np
import pytest

from oracle import packed as K


def test_tables():
    assert K.TABLES["e2m1"].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    t = K.TABLES["e4m3"]
    assert len(t) == 127 and t[-1] == 448 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6
    assert K.TABLES["int8"][-1] == 127 / 64


@pytest.mark.parametrize("fmt,value,byte", [
    ("e4m3", 448.0, 127), ("e4m3", 448.5, 128), ("e4m3", 224.0, 126), ("e4m3", 1.0, 119),
    ("int8", 127 / 64, 127), ("int8", 2.0, 128), ("int8", 1.0, 127), ("int8", 0.9921875, 126),
    ("e2m1", 6.0, 127), ("e2m1", 6.0625, 128), ("e2m1", 3.0, 126), ("e2m1", 1.0, 125)])
def test_scale_rule(fmt, value, byte):
    x = np.zeros((1, 32))
    x[0, 5] = -value
    codes, s, v = K.quantise(x, fmt)
    assert s[0, 0] == byte
    assert abs(v[0, 5] + value) <= value * 2.0 ** -3


@pytest.mark.parametrize("fmt,pairs", [
    ("e2m1", [(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0),
              (0.2500001, 0.5), (-2.5, -2.0)]),
    ("int8", [(0.5 / 64, 0.0), (1.5 / 64, 2 / 64), (-2.5 / 64, -2 / 64), (2.51 / 64, 3 / 64)]),
    ("e4m3", [(17.0, 16.0), (19.0, 20.0), (2.0 ** -10, 0.0), (3 * 2.0 ** -10, 2.0 ** -8), (-17.0, -16.0)])])
def test_ties_go_to_the_even_code(fmt, pairs):
    x = np.zeros((len(pairs), 32))
    x[:, 0] = K.LARGEST[fmt]  # scale byte 127: values stand for themselves
    x[:, 1] = [p[0] for p in pairs]
    _, s, v = K.quantise(x, fmt)
    assert (s == 127).all()
    assert v[:, 1].tolist() == [p[1] for p in pairs]


def test_clamps_and_non_finite_blocks():
    # the largest finite values: (1.875, 127/64, 1.5) 2^127 against nearly 2^128
    worst = {"e4m3": 1 / 16, "int8": 1 / 128, "e2m1": 1 / 4}
    for fmt in K.TABLES:
        x = np.zeros((5, 64))
        x[1, 3] = 1e-40                      # below the smallest scale: zero
        x[2, 40] = np.inf
        x[3, 1] = np.nan
        x[4, 0] = np.finfo(np.float32).max   # the largest scale still holds it
        codes, s, v = K.quantise(x, fmt)
        assert (s[0] == K.LO[fmt]).all() and (codes[0] == 0).all()
        assert s[1, 0] == K.LO[fmt] and v[1, 3] == 0
        assert s[2].tolist() == [K.LO[fmt], 255] and np.isnan(v[2, 32:]).all() and (v[2, :32] == 0).all()
        assert s[3, 0] == 255 and (codes[3, :32] == 0).all()
        assert s[4, 0] <= 254 and abs(v[4, 0] / x[4, 0] - 1) <= worst[fmt]
        assert v[4, 0] < 2.0 ** 128


def test_error_bounds_and_short_last_block():
    g = np.random.Generator(np.random.PCG64(1))
    x = g.standard_normal((200, 72)) * np.exp(g.standard_normal((200, 1)) * 8)
    for fmt in ("e4m3", "int8", "e2m1"):
        codes, s, v = K.quantise(x, fmt)
        assert codes.shape == x.shape and s.shape == (200, 3)
        amax = np.stack([np.abs(x[:, i:i + 32]).max(1) for i in (0, 32, 64)], 1)
        amax = np.repeat(amax, 32, 1)[:, :72]
        err = np.abs(v - x)
        if fmt == "e4m3":
            big = np.abs(x) > 2.0 ** -13 * amax
            assert (err[big] <= 2.0 ** -4 * np.abs(x[big])).all()
        elif fmt == "int8":
            assert (err <= amax / 127).all()
        else:
            assert (err <= amax / 3).all()
        # what was stored stores again unchanged
        assert (K.quantise(v, fmt)[2] == v).all()


def test_values4_reads_what_quantise_wrote():
    g = np.random.Generator(np.random.PCG64(2))
    x = g.standard_normal((6, 64))
    codes, s, v = K.quantise(x, "e2m1")
    assert (K.values4(K.pack4(codes), s) == v).all()
