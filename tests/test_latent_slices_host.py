"""kda_rotary from some columns of the heads into other columns of the same heads: nothing
overlaps, whether rows follow one another without a gap or not.  No GPU: what passes the
checks ends at the launch without a device (-7)."""
import ctypes
import itertools
import os
import random

import pytest
import torch

from gated_delta_rule_55_amd import _abi
from gated_delta_rule_55_amd import _abi_latent as al

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0 or not os.path.exists(_abi.LIB_PATH),
                                reason="fake-pointer checks run without a GPU, on the built library")
X = 0x1000000


def rotary(**kw):
    d = al.make(al.RotaryDesc, **dict(dict(dtype=2, n_heads=4, dim=64, t_total=9, x=X, positions=0x3000000,
                                           frequencies=0x3001000), **kw))
    return al.lib().kda_rotary(ctypes.byref(d), None)


@pytest.mark.parametrize("row", [0, 4 * 192, 4 * 192 + 576, 4 * 192 + 8])
@pytest.mark.parametrize("heads,tokens", [(4, 9), (1, 9), (4, 1)])
def test_other_columns_of_the_same_heads(row, heads, tokens):
    s = dict(n_heads=heads, t_total=tokens, x_stride=row, y_stride=row, x_head_stride=192, y_head_stride=192)
    for column in (64, 72, 128):
        assert rotary(**s, y=X + 2 * column) == -7
        assert rotary(**s, y=X, x=X + 2 * column) == -7
    for column in (8, 56):
        assert rotary(**s, y=X + 2 * column) == -9
        assert rotary(**s, y=X, x=X + 2 * column) == -9
    if tokens == 1:
        assert rotary(**dict(s, y_stride=5120), y=X + 2 * 64) == -7 and rotary(**dict(s, y_stride=5120), y=X + 2 * 56) == -9
    # a head further: the same columns of the heads behind the first
    assert rotary(**s, y=X + 2 * 192) == (-9 if heads > 1 or (tokens > 1 and row == 0) else -7)


def places(tokens, heads, row, head, d, at):
    return {at + t * row + h * head + i for t in range(tokens) for h in range(heads) for i in range(0, d, 8)}


def test_refused_where_they_overlap_and_nowhere_else():
    """Against the places themselves, in steps of 16 bytes; equal strides on both sides."""
    r = random.Random(1)
    passed = 0
    for _ in range(4000):
        T, H, d = r.choice([1, 2, 3]), r.choice([1, 2, 3]), 16 * r.randint(1, 3)
        head = d + 8 * r.randint(0, 12)
        row = (H - 1) * head + d + 8 * r.randint(0, 20)
        at = 8 * r.randint(-120, 120)
        if at == 0:
            continue
        apart = not (places(T, H, row, head, d, 0) & places(T, H, row, head, d, at))
        s = dict(dim=d, n_heads=H, t_total=T, x_stride=row, y_stride=row, x_head_stride=head, y_head_stride=head)
        assert rotary(**s, y=X + 2 * at) == (-7 if apart else -9)
        passed += apart
    assert 500 < passed < 3500
