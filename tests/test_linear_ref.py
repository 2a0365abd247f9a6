"""The tests' own forms of the mask and the activations, pinned (CPU)."""
import numpy as np
import pytest
import torch

from tests import linear_ref as ref


@pytest.mark.parametrize("ctr,key,out", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])])
def test_philox_known_answers(ctr, key, out):
    """the generator's published known answers (ten rounds)"""
    got = ref.philox([np.array([c], np.uint64) for c in ctr], key)
    assert [int(g[0]) for g in got] == out


def test_every_column_has_bits_of_its_own():
    """columns of a group of 32 take 4 blocks x 4 words x 2 halves, once each"""
    u = ref.bits16(3, 64, 5, 9, 2)
    for r in range(3):
        for group in range(2):
            words = [ref.philox([np.array([group * 4 + b], np.uint64),
                                 np.array([2 + r], np.uint64), np.array([9], np.uint64),
                                 np.array([0], np.uint64)], (5, 0)) for b in range(4)]
            halves = sorted(int(w[0]) >> (16 * h) & 0xFFFF for b in words for w in b for h in (0, 1))
            assert sorted(u[r, group * 32:group * 32 + 32]) == halves


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_are_the_derivatives(act):
    v = torch.linspace(-6, 6, 1001, dtype=torch.float64) + 1e-3
    h = 1e-6
    diff = (ref.act64(v + h, act)[0] - ref.act64(v - h, act)[0]) / (2 * h)
    assert torch.allclose(ref.act64(v, act)[1], diff, atol=1e-8)
    f = {"relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh"),
         "silu": torch.nn.functional.silu}[act]
    assert torch.allclose(ref.act64(v, act)[0], f(v), atol=1e-12)
