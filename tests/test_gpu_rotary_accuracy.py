"""How far sine, cosine and the angle of the rotary calls are off, seen in fp32:
the scale of a key appended with scales per token is its largest magnitude after
the turn over 448, before anything is rounded to bf16 or e4m3."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a step of fp32, relative
# Sine and cosine: the rounding of a number below 1 is within 0.5 U.  The rest of
# at most 0.02455 rad carries three roundings (0.074 U), the table's entry times
# it is rounded once in its series and once in the sum (0.025 U each), and what the
# series leaves out is 7.4e-11 (0.0013 U): 0.63 U with the second-order ones.
TABLE = 0.65 * U
# 2 pi to 200 bits as a whole number of 2^-200 (pi = 3.14159265358979323846264338327950288419716939937510582097494459)
PI_DIGITS = 314159265358979323846264338327950288419716939937510582097494459
TWO_PI_200 = (2 * PI_DIGITS << 200) // 10 ** 62


@pytest.fixture(scope="module")
def pf():
    import paged_fp8_kv_02_gb300 as m
    m.load()
    return m


def angles(freq, pos):
    """Fractions of a turn of position * frequency, in whole numbers: float64
    [T][pairs] in [0, 1), off by 2^-54."""
    out = np.empty((len(pos), len(freq)))
    for j, f in enumerate(freq):
        n, d = float(f).as_integer_ratio()
        turn = (n << 400) // (d * TWO_PI_200)   # of 2^-200: f / 2 pi
        for i, p in enumerate(pos):
            out[i, j] = (int(p) * turn % (1 << 200) >> 140) / 2.0 ** 60
    return out


def largest(pf, freq, pos, x, y):
    """max(|x'|, |y'|) as the library has it in fp32, over 448 and rounded, for
    the pair (x, y) turned by every position and frequency: float64 [T][pairs].
    Head h holds pair h alone."""
    import torch
    T, n, P = len(pos), len(freq), 16
    assert n == 64
    k = torch.zeros(T, n, 2 * n, dtype=torch.bfloat16, device="cuda")
    h = torch.arange(n, device="cuda")
    k[:, h, h], k[:, h, h + n] = x, y
    pages = -(-T // P)
    cache = torch.zeros(pages, n, P, 2 * n, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages, n, P, device="cuda")
    pf.rotary_append_fp8(None, None, k, None, cache, None, torch.arange(T, device="cuda"),
                         torch.from_numpy(np.asarray(pos, np.int32)).cuda(), pf.Rotary(freq), pf.SCALE_TOKEN, scales)
    return scales.double().permute(0, 2, 1).reshape(-1, n)[:T].cpu().numpy() * 448


@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("span", [4096, 2 ** 31 - 1])
def test_sine_cosine_and_angle(pf, base, span):
    freq = base ** (-np.arange(64) / 64)
    rng = np.random.default_rng(int(base) + span % 1000)
    pos = np.concatenate([[0, 1, -1, span, -span - (span == 2 ** 31 - 1)], rng.integers(-span, span, 2043)]).astype(np.int64)
    phi = 2 * np.pi * angles(freq, pos)
    c, s = np.cos(phi), np.sin(phi)
    # the stated error of the angle: 2^-64 of a turn per position and 2^-52 of the angle; sine and cosine move by no more
    turn = np.abs(pos)[:, None] * (2 * np.pi * 2.0 ** -64 + 2.0 ** -52 * freq)
    one = TABLE + turn + 1e-15   # and the reference's own
    # (1, 0) turns to (cos, sin): the larger one, and the division's rounding
    want = np.maximum(np.abs(c), np.abs(s))
    got = largest(pf, freq, pos, 1.0, 0.0)
    assert np.all(np.abs(got - want) <= one + want * U), np.max((np.abs(got - want) - want * U - turn) / U)
    # (1, 1) turns to cos - sin, cos + sin: |cos| + |sin|, rounded once in 1 .. 2 (U) and by the division
    want = np.abs(c) + np.abs(s)
    got = largest(pf, freq, pos, 1.0, 1.0)
    assert np.all(np.abs(got - want) <= 2 * one + U + want * U)


def test_sine_and_cosine_all_around(pf):
    """Angles spread evenly over the turn, and next to the borders of the 128
    parts that the table has."""
    step = 2.0 ** -32   # positions count 2^-32 of a turn
    f = 2 * np.pi * step * (1 - 2.0 ** -20 * np.arange(64))
    even = np.arange(-2 ** 31, 2 ** 31, 2 ** 20 + 12345)
    at = (np.arange(-64, 64) * 2 ** 25 + 2 ** 24)[:, None] + np.array([-2, -1, 0, 1, 2])
    mid = (np.arange(-64, 64) * 2 ** 25)[:, None] + np.array([-1, 0, 1])
    pos = np.concatenate([even, at.ravel(), mid.ravel()])
    pos = np.clip(pos, -2 ** 31, 2 ** 31 - 1)
    phi = 2 * np.pi * angles(f, pos)
    want = np.maximum(np.abs(np.cos(phi)), np.abs(np.sin(phi)))
    got = largest(pf, f, pos, 1.0, 0.0)
    turn = np.abs(pos)[:, None] * (2 * np.pi * 2.0 ** -64 + 2.0 ** -52 * f)
    assert np.all(np.abs(got - want) <= TABLE + turn + 1e-15 + want * U)
