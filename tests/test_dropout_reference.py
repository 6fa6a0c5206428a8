"""Pins of the mask reference: the generator's published known answers, and the mask's frequency."""
import numpy as np
import pytest

from tests.dropout_reference import kept, philox4x32_10, threshold


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_gives_the_published_answers(counter, key, want):
    got = philox4x32_10(np.array([counter], dtype=np.uint64), key)
    assert [int(v) for v in got[0]] == list(want)


def test_frequency_and_independence_of_offsets():
    n = 1 << 18
    a, b = kept(n, 0.3, 5, 1), kept(n, 0.3, 5, 2)
    q = threshold(0.3) / 65536
    sd = (q * (1 - q) / n) ** 0.5
    assert abs((~a).mean() - q) < 5 * sd and abs((~b).mean() - q) < 5 * sd
    assert abs((~a & ~b).mean() - q * q) < 5 * (q * q * (1 - q * q) / n) ** 0.5
    assert (kept(n // 2, 0.3, 5, 1, first=n // 2) == a[n // 2:]).all()
    assert kept(100, 0.0, 5, 1).all()
