"""Limits of the decoder operators that need no GPU: how whole numbers reach
the library, sizes at the ends of their ranges, and the memory that a call
asks for."""
import enum
import time

import numpy as np
import pytest
import torch

from sparse_attention_banded_b200 import build, lf


@pytest.fixture(scope="module")
def L():
    build.build()
    return lf.lib()


class Window(enum.IntEnum):
    SHORT = 4


def _qkv(L=8):
    return (torch.zeros(1, 4, L, 64, dtype=torch.float16), torch.zeros(1, 2, L, 64, dtype=torch.float16))


@pytest.mark.timeout(30)
@pytest.mark.parametrize("w", [4, np.int64(4), np.int32(4), Window.SHORT, True, torch.tensor(4)])
def test_any_whole_number_is_taken_at_once(w):
    """Numbers other than Python's own int are converted, not searched for in
    a range of 2^32 (the call then goes on to refuse CPU tensors)."""
    q, k = _qkv()
    t0 = time.monotonic()
    with pytest.raises(ValueError, match="CUDA"):
        lf.lf_window_attention_forward(q, k, k, w, sinks=w)
    assert time.monotonic() - t0 < 5


@pytest.mark.timeout(30)
@pytest.mark.parametrize("w,error", [(4.0, TypeError), (0.5, TypeError), ("4", TypeError), (None, TypeError),
                                     (np.int64(1 << 31), ValueError), (-(1 << 31) - 1, ValueError)])
def test_other_numbers_are_refused_at_once(w, error):
    q, k = _qkv()
    t0 = time.monotonic()
    with pytest.raises(error):
        lf.lf_window_attention_forward(q, k, k, w)
    with pytest.raises(error):
        lf.lf_window_attention_forward(q, k, k, 4, sinks=w)
    assert time.monotonic() - t0 < 5
