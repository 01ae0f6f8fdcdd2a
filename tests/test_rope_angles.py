"""The rotary step's frequencies and angles against whole numbers: pi by Machin's formula, no floating point."""
import ctypes
import math
import random
from fractions import Fraction

import pytest
import torch

import chunked_recurrence_gb300 as crg


def _pi(bits):
    one = 1 << (bits + 32)

    def atan_inverse(x):
        term, total, n = one // x, one // x, 3
        while term:
            term //= x * x
            total += -(term // n) if n % 4 == 3 else term // n
            n += 2
        return total
    return Fraction(4 * (4 * atan_inverse(5) - atan_inverse(239)), one)


TWO_PI = 2 * _pi(1400)


def _words(inv):
    return [w % 2 ** 64 for w in crg.gdn_rope_freqs(torch.tensor(inv, dtype=torch.float64), device="cpu").tolist()]


def _frequencies():
    rng = random.Random(3)
    inv = [1.0, -1.0, 1e-4, 0.3, 6.283185307179586, math.pi, 2.0 ** 52 + 1, -(2.0 ** 53 - 1), 2.0 ** -200, 5e-324, 0.0,
           2.0 ** -63, 2.0 ** -62, 2.0 ** -61]
    inv += [10000.0 ** (-2 * i / d) for d in (64, 128) for i in range(d // 2)]
    return inv + [rng.choice([-1, 1]) * rng.random() * 2.0 ** rng.randint(-70, 53) for _ in range(500)]


def test_words_are_the_nearest():
    inv = _frequencies()
    for x, w in zip(inv, _words(inv)):
        turns = Fraction(x) / TWO_PI * 2 ** 64
        off = abs(turns - w) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2), x


def test_angles_at_far_positions():
    """Against the true angle, for every position of 64 bits: 2^-65 turns a position."""
    rng = random.Random(4)
    inv = _frequencies()
    for x, w in zip(inv, _words(inv)):
        for p in (1, 10 ** 6, 2 ** 31, -7, rng.randint(-2 ** 63, 2 ** 63 - 1)):
            off = abs(Fraction(p * w, 2 ** 64) - p * Fraction(x) / TWO_PI) % 1
            assert min(off, 1 - off) <= abs(p) * Fraction(1, 2 ** 65), (x, p)


def test_refusals():
    words = (ctypes.c_uint64 * 1)()
    for bad in (math.inf, -math.inf, math.nan, 2.0 ** 53, -(2.0 ** 60)):
        assert crg.load().gdn_rope_freqs((ctypes.c_double * 1)(bad), 1, words) == 1


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("inter", [False, True])
def test_turns_at_far_positions(inter):
    """The kernel's cos and sin at the true angle.  Off by: the angle cut to 2^-32 turns, |p| 2^-65 turns of the
    frequency, and 2^-23 for each of cos and sin, their products and their sum (1 each): 2^-21 and the angle's part
    times 2 (|cos| + |sin|)."""
    inv = crg.gdn_rope_inv_freq(64)
    pos = [0, 1, 10 ** 6, 2 ** 31, 2 ** 40 + 3, -(2 ** 40), 2 ** 45 - 9]
    q = torch.ones((len(pos), 1, 64), device="cuda")
    out, _ = crg.gdn_rope(q, None, torch.tensor(pos, device="cuda"), crg.gdn_rope_freqs(inv), inter)
    out = out.double().cpu()
    for t, p in enumerate(pos):
        angle_off = 2 * math.pi * (2.0 ** -32 + abs(p) * 2.0 ** -65)
        for i, x in enumerate(inv.tolist()):
            turns = (p * Fraction(x) / TWO_PI) % 1
            a = 2 * math.pi * float(turns)
            y1, y2 = (out[t, 0, 2 * i], out[t, 0, 2 * i + 1]) if inter else (out[t, 0, i], out[t, 0, 32 + i])
            assert abs(y1.item() - (math.cos(a) - math.sin(a))) <= 2.0 ** -21 + 2 * angle_off, (p, i)
            assert abs(y2.item() - (math.cos(a) + math.sin(a))) <= 2.0 ** -21 + 2 * angle_off, (p, i)


def test_tokens_too_wide_are_refused():
    """Places within a token are 32-bit numbers in the kernel."""
    fake = ctypes.c_void_p(0x10000)  # never dereferenced
    crg.load()

    def call(Hq, Hk, D):
        return crg.load().gdn_rope(fake, fake, fake, fake, 1, 1, Hq, Hk, D, 2, 0, 0, 0, 0, 1.0, 0, fake, fake, None)
    for Hq, Hk, D in ((1 << 24, 0, 128), (1 << 22, 1 << 22, 64), (0, 2 ** 31 - 1, 1), (2 ** 31 - 1, 2 ** 31 - 1, 256)):
        assert call(Hq, Hk, max(D, 2)) == 2, (Hq, Hk, D)
