"""The marks of latent_marks show a lost or doubled tile of keys, wherever it lies, to
the bounds that the GPU tests use: planted in the oracle's sums, without a GPU."""
import numpy as np
import pytest
import torch

from latent_cases import BF, check_attention
from latent_marks import COURSES, FACTORS, scores, values


def attention(w, v):
    """w [R, L] unnormalised weights: o [R, columns]."""
    return w @ v / w.sum(1, keepdims=True)


@pytest.mark.parametrize("dtype,length,columns,tile", [(BF, 32768, 512, 64), (BF, 8192, 128, 64), (BF, 8000, 256, 64),
                                                       (torch.float32, 16384, 512, 32), (torch.float32, 3000, 128, 64)])
@pytest.mark.parametrize("course", COURSES)
def test_every_tile_is_seen(dtype, length, columns, tile, course):
    s, v = scores(course, length), values(length, columns)
    assert np.array_equal(torch.from_numpy(s).bfloat16().double().numpy(), s)
    w = np.exp(np.outer(FACTORS, s))
    o = attention(w, v)
    ref = (o, o, np.abs(np.outer(FACTORS, s)).max(1))
    check_attention(torch.from_numpy(o).to(dtype), ref, length, 576)   # the right answer, rounded
    num, den = w @ v, w.sum(1, keepdims=True)
    for begin in range(0, length, tile):
        part = slice(begin, min(begin + tile, length))
        n, d = w[:, part] @ v[part], w[:, part].sum(1, keepdims=True)
        for sign in (-1, 1):
            wrong = torch.from_numpy((num + sign * n) / (den + sign * d)).to(dtype)
            with pytest.raises(AssertionError):
                check_attention(wrong, ref, length, 576)
