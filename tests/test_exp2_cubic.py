"""The prefix decode's FMA-pipe exp2 (exp2_cubic2 in csrc/decode_prefix.cuh), checked on
the CPU: its coefficients are those of the committed fit with degree 3, and its float32
steps stay within the fit's error over the range of exponents that the softmax feeds
(at most 8, the growth after which the running reference moves; clamped at -126).  Also
the 32-bit form of the even split."""
import os
import random
import re

import numpy as np

from llama_gqa_causal_b200.csrc.fit_exp2_poly import remez_rel

SOURCE = os.path.join(os.path.dirname(__file__), "..", "llama_gqa_causal_b200", "csrc",
                      "decode_prefix.cuh")


def _coefficients():
    src = open(SOURCE).read()
    body = src[src.index("void exp2_cubic2("):]
    body = body[:body.index("\n}\n")]
    assert "fmaxf(x0, -126.f)" in body and "fmaxf(x1, -126.f)" in body
    vals = dict(re.findall(r"\b(c\d) = ([0-9.eE+-]+)f", body))
    return np.array([float(vals[f"c{i}"]) for i in range(len(vals))], dtype=np.float32)


def _fma32(a, b, c):
    # one rounding of a * b + c to float32 (the product of two float32 is exact in float64)
    return (a.astype(np.float64) * b.astype(np.float64) + c.astype(np.float64)).astype(np.float32)


def _exp2(x, c):
    x = np.maximum(x.astype(np.float32), np.float32(-126.0))
    k = np.float32(12582912.0)
    t = (x + k).astype(np.float32)
    f = _fma32((t - k).astype(np.float32), np.float32(-1.0), x)
    q = np.full_like(f, c[3])
    for i in (2, 1, 0):
        q = _fma32(q, f, np.full_like(f, c[i]))
    bits = q.view(np.int32).astype(np.int64) + (t.view(np.int32).astype(np.int64) << 23)
    return (bits & 0xFFFFFFFF).astype(np.uint32).view(np.int32).view(np.float32)


def test_coefficients_are_the_fit():
    c = _coefficients()
    fit, err = remez_rel(3)
    assert len(c) == 4 and np.array_equal(c, fit.astype(np.float32)) and err < 7.6e-5


def test_relative_error_over_the_input_range():
    """The fit's error, and half a step (2^-24) for each of three products and sums of
    size about one and for the coefficients."""
    x = np.concatenate([np.linspace(-125.5, 8.0, 2_000_001, dtype=np.float32),
                        np.arange(-125, 9, dtype=np.float32),
                        np.arange(-125, 8, dtype=np.float32) + 0.5])
    y, ref = _exp2(x, _coefficients()).astype(np.float64), np.exp2(x.astype(np.float64))
    assert (np.abs(y - ref) / ref).max() < 7.6e-5 + 4 * 2.0 ** -24


def test_far_below_is_tiny_and_not_negative():
    y = _exp2(np.array([-126.0, -127.0, -1e4, -3e38, -np.inf], dtype=np.float32), _coefficients())
    assert (y >= 0).all() and (y < 2.0 ** -125).all()


def test_even_split_in_32_bits():
    """i n // g = i (n // g) + i (n % g) // g, with nothing past 31 bits for g up to 12 x 148."""
    rng = random.Random(0)
    for _ in range(20000):
        g = rng.randint(1, 12 * 148)
        n = rng.randint(g, 2 ** 31 - 1) if rng.random() < 0.5 else rng.randint(g, 4 * g)
        i = rng.randint(0, g)
        each, rest = divmod(n, g)
        assert i * each <= 2 ** 31 - 1 and i * rest <= 2 ** 31 - 1
        assert i * n // g == i * each + i * rest // g
