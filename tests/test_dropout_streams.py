"""Which calls of the dropout share a mask (CPU): the stream is offset plus
step, so neighbouring offsets meet as the step counter moves; offsets 2^32
apart do not.  The documentation says both."""
import os

import numpy as np

import zero_sharded_mixed_flatten_amd as zs
from tests import linear_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_neighbouring_offsets_meet_in_later_steps():
    layer0_step6 = ref.bits16(5, 100, 7, 0 + 6)
    assert np.array_equal(ref.bits16(5, 100, 7, 1 + 5), layer0_step6)


def test_offsets_apart_by_more_than_the_steps_do_not():
    """every layer and step of a grid draws bits of its own: the first rows'
    64 bits are all different"""
    seen = set()
    for layer in range(8):
        for step in range(1, 33):
            seen.add(tuple(ref.bits16(1, 4, 7, (layer << 32) + step)[0]))
    assert len(seen) == 8 * 32


def test_the_rule_stands_where_users_read_it():
    header = open(os.path.join(ROOT, "include", "zero_linear.h"), encoding="utf-8").read()
    part = " ".join(header[header.index("/* Dropout D"):header.index("zero_dropout_params {")]
                    .replace("*", " ").split())
    assert "offset + step" in part and "multiples of 2^32" in part and "different seeds" in part
    assert "<< 32" in zs.ZeroDropout.__doc__ and "defaults" in zs.ZeroDropout.__doc__
    readme = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    assert "layer << 32" in readme
