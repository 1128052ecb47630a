"""The 4-bit record of the tests' reference, against exact fractions and by hand.

Every step of the quantisation is one operation rounded to its type, so it can be done in
whole fractions with one rounding rule, apart from any floating-point library."""
import random
from fractions import Fraction

import pytest
import torch

from _q4_ref import records, values

LOW, BITS = {"fp16": -24, "fp32": -149}, {"fp16": 11, "fp32": 24}


def rounded(x, kind):
    """Fraction x to the nearest number of the type, half to even (no overflow here)."""
    if x == 0:
        return x
    e = 0
    while abs(x) >= Fraction(2) ** (e + 1):
        e += 1
    while abs(x) < Fraction(2) ** e:
        e -= 1
    step = Fraction(2) ** max(e + 1 - BITS[kind], LOW[kind])
    return round(x / step) * step  # (Python rounds halves of fractions to even)


def half_bits(x):
    """The two bytes of Fraction x, a number of fp16."""
    s, x = (0x8000, -x) if x < 0 else (0, x)
    if x < Fraction(2) ** -14:
        n = int(x * 2 ** 24)
    else:
        e = 15
        while x < Fraction(2) ** e:
            e -= 1
        n = (e + 15 << 10) + int((x / Fraction(2) ** e - 1) * 1024)
    return [(s + n) & 255, (s + n) >> 8]


def record(row):
    D = len(row)
    codes, scales, least = [0] * D, [], []
    clamp = lambda x, a, b: max(Fraction(a), min(Fraction(b), x))  # noqa: E731
    fifteenth = rounded(Fraction(1, 15), "fp32")
    for g in range(4):
        x = row[g * D // 4:(g + 1) * D // 4]
        lo = rounded(clamp(min(x), -65504, 65504), "fp16")
        sc = rounded(clamp(rounded(rounded(max(x) - lo, "fp32") * fifteenth, "fp32"), 0, 65504), "fp16")
        least.append(lo)
        scales.append(sc)
        for i, v in enumerate(x):
            u = rounded(rounded(v - lo, "fp32") / sc, "fp32") if sc else Fraction(0)
            codes[g * D // 4 + i] = int(clamp(Fraction(round(u)), 0, 15))
    pairs = [codes[2 * i] + 16 * codes[2 * i + 1] for i in range(D // 2)]
    if D == 64:  # the bytes of groups 0 and 1 by turns, then of 2 and 3
        pairs = [pairs[16 * (i // 16) + 8 * (i % 2) + i % 16 // 2] for i in range(32)]
    return pairs + [b for x in scales + least for b in half_bits(x)]


@pytest.mark.parametrize("D", [64, 128])
def test_records_against_fractions(D):
    rng = random.Random(D)
    rows = []
    for size in (1e-6, 1e-3, 1.0, 37.0, 3e4):
        for at in (0.0, 1.0, -20.0):
            rows.append([size * (rng.gauss(0, 1) + at) for _ in range(D)])
    rows += [[0.0] * D, [-2.5] * D, [float(i % 16) for i in range(D)], [(i % 31) / 2 - 8 for i in range(D)],
             [1000.0 if i % 9 == 0 else rng.random() for i in range(D)]]
    x = torch.tensor(rows, dtype=torch.float32).clamp(-6e4, 6e4)
    want = [record([Fraction(v) for v in row]) for row in x.double().tolist()]
    assert records(x).tolist() == want


def test_a_record_by_hand():
    """Features 0 .. 15 twice in each group of 32: least 0, scale 1, codes as they are; the last group is
    -4 .. 3.5 in halves: least -4, scale 0.5."""
    row = [float(i % 16) for i in range(96)] + [i % 16 / 2 - 4 for i in range(32)]
    pairs = [0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe]
    one, half, minus_four = [0x00, 0x3c], [0x00, 0x38], [0x00, 0xc4]
    want = pairs * 8 + one * 3 + half + [0, 0] * 3 + minus_four
    rec = records(torch.tensor([row]))
    assert rec[0].tolist() == want
    x, _ = values(rec)
    assert x[0].tolist() == row


def test_a_short_record_by_hand():
    """64 features: groups of 16, whose bytes come by turns. Group g has its features' places plus 100 g (least
    100 g, scale 1)."""
    row = [float(i % 16 + 100 * (i // 16)) for i in range(64)]
    pairs = [0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe]
    turns = [b for p in pairs for b in (p, p)]
    want = turns * 2 + [0x00, 0x3c] * 4 + [0x00, 0x00, 0x40, 0x56, 0x40, 0x5a, 0xb0, 0x5c]
    rec = records(torch.tensor([row]))
    assert rec[0].tolist() == want
    assert values(rec)[0][0].tolist() == row
    assert values(torch.tensor([[0x21, 0x43] + [0] * 30 + want[32:]], dtype=torch.uint8))[0][0, [0, 1, 16, 17]].tolist() == \
        [1.0, 2.0, 103.0, 104.0]
