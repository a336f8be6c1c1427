"""The counter-based generator of dropout, in plain integers: its published answers, and that the plain form of
the measured cases and the one that the GPU tests compare with draw the same numbers."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LOW = 0xFFFFFFFF


def philox(counter, key):
    """Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, 2011) of four and two 32-bit words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [b >> 32 ^ c[1] ^ k[0], b & LOW, a >> 32 ^ c[3] ^ k[1], a & LOW]
        k = [k[0] + 0x9E3779B9 & LOW, k[1] + 0xBB67AE85 & LOW]
    return c


@pytest.mark.parametrize("counter,key,want", [  # the answers published with the generator
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((LOW, LOW, LOW, LOW), (LOW, LOW), (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))])
def test_published_answers(counter, key, want):
    assert tuple(philox(counter, key)) == want


RNGS = [(0, 0, 0), (1234567890123456789, 41, 7), (-3, 2 ** 33 + 5, 2 ** 32 - 1), (2 ** 40 + 9, -1, 3)]


def of_element(i, seed, stream, site):
    block = i // 4
    return philox((block & LOW, block >> 32 & LOW, stream & LOW, (stream >> 32) + site & LOW),
                  (seed & LOW, seed >> 32 & LOW))[i % 4]


@pytest.mark.parametrize("seed,stream,site", RNGS)
def test_the_gpu_tests_numbers(seed, stream, site):
    from test_gpu_stack import words
    assert [int(v) for v in words(70, seed, stream, site)] == [of_element(i, seed, stream, site) for i in range(70)]
    for start in (2 ** 32 - 8, 2 ** 34 - 8, 2 ** 34, 5 * 2 ** 35 + 16):
        got = words(16, seed, stream, site, start)
        assert [int(v) for v in got] == [of_element(start + i, seed, stream, site) for i in range(16)]


@pytest.mark.parametrize("seed,stream,site", RNGS)
def test_the_measured_cases_numbers(seed, stream, site):
    spec = importlib.util.spec_from_file_location("cases", os.path.join(ROOT, "perf", "more_operators.py"))
    cases = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cases)
    got = cases.random_words(70, torch.tensor([seed, stream]), site).tolist()
    assert got == [of_element(i, seed, stream, site) for i in range(70)]
