"""Calls of latent attention on a single token, whose row strides say nothing: the callers
leave them out or make them up, and a call in place is one all the same.  No GPU: what
passes the checks ends at the launch without a device (-7)."""
import ctypes
import os

import pytest
import torch

from gated_delta_rule_55_amd import _abi
from gated_delta_rule_55_amd import _abi_latent as al

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0 or not os.path.exists(_abi.LIB_PATH),
                                reason="fake-pointer checks run without a GPU, on the built library")
ROW = 0x1000000
APPEND = dict(dtype=2, n_seqs=1, dc=512, dr=64, page_size=64, max_pages=8, n_pages=20, eps=1e-6, t_total=1, latent=ROW,
              k_pe=ROW + 1024, rows_out=ROW, cache=0x2000000, weight=0x4000000, frequencies=0x4100000,
              block_table=0x6000000, seq_lens=0x6001000)


def append(**over):
    d = al.make(al.LatentAppendDesc, **dict(APPEND, **over))
    return al.lib().kda_latent_append(ctypes.byref(d), None)


# as the true slices have them, as none, as each dense by itself, and as a program may fill them
STRIDES = [(576, 576, 576), (0, 0, 0), (512, 64, 576), (640, 576, 0), (1024, 128, 2048)]


@pytest.mark.parametrize("strides", STRIDES)
@pytest.mark.parametrize("cu", [None, 0x6002000])
def test_append_of_one_token_in_place(strides, cu):
    lat, pe, out = strides
    kw = dict(latent_stride=lat, k_pe_stride=pe, rows_out_stride=out, cu_seqlens=cu)
    assert append(**kw) == -7
    # what is not in place stays refused: a row further, the parts in another order, one input elsewhere
    assert append(**kw, k_pe=ROW + 1040) == -9
    assert append(**kw, rows_out=ROW + 16) == -9
    assert append(**kw, latent=ROW + 128, k_pe=ROW) == -9
    assert append(**kw, latent=0x1800000) == -9
    assert append(**kw, k_pe=0x1800000) == -9


def test_append_of_two_tokens_needs_their_strides():
    two = dict(t_total=2, n_seqs=2)
    assert append(**two, latent_stride=576, k_pe_stride=576, rows_out_stride=576) == -7
    for lat, pe, out in STRIDES[1:]:
        assert append(**two, latent_stride=lat, k_pe_stride=pe, rows_out_stride=out) == -9


ROTARY = dict(dtype=2, n_heads=4, dim=64, rotary=1, t_total=9, x=ROW, y=ROW, positions=0x3000000, frequencies=0x3001000)


@pytest.mark.parametrize("over,status", [
    (dict(t_total=1, x_stride=0, y_stride=320), -7), (dict(t_total=1, x_stride=768, y_stride=0), -7),
    (dict(t_total=1, n_heads=1, x_head_stride=128, y_stride=640), -7),
    (dict(n_heads=1, x_stride=192, y_stride=192, x_head_stride=64, y_head_stride=192), -7),
    (dict(t_total=1, x_head_stride=128), -9),                                # heads that do not meet
    (dict(t_total=1, y_stride=320, y=ROW + 16), -9),
    (dict(n_heads=1, x_stride=192, y_stride=256), -9), (dict(x_stride=320), -9),
])
def test_rotary_in_place(over, status):
    d = al.make(al.RotaryDesc, **dict(ROTARY, **over))
    assert al.lib().kda_rotary(ctypes.byref(d), None) == status
