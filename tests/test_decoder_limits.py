"""Limits of the decoder operators that need no GPU: how whole numbers reach
the library, sizes at the ends of their ranges, and the memory that a call
asks for."""
import enum
import time

import numpy as np
import pytest
import torch

from sparse_attention_banded_b200 import build, lf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lf.lib()


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


def _wide(*shape, dtype=torch.float16):
    """A tensor of any shape over one element."""
    return torch.zeros((), dtype=dtype).expand(shape)


BIG = (1 << 32) + 8  # cut to 32 bits this would be 8


def test_sizes_past_32_bits_are_refused():
    """A size that the C interface's int cannot hold is an error, not another
    size."""
    i32 = torch.int32
    with pytest.raises(ValueError, match="int32"):
        lf.lf_window_attention_forward(_wide(BIG, 1, 64), _wide(BIG, 1, 64), _wide(BIG, 1, 64), 4,
                                       cu_seqlens=torch.zeros(2, dtype=i32))
    q = _wide(1, 1, BIG, 64)
    with pytest.raises(ValueError, match="int32"):
        lf.lf_window_attention_forward(q, q, q, 4)
    with pytest.raises(ValueError, match="int32"):
        lf.lf_window_attention_backward(q, q, q, _wide(1, BIG, 64), _wide(1, 1, BIG, dtype=torch.float32),
                                        _wide(1, BIG, 64), 4)
    q, cache, cu, kv = _wide(1, 1, 64), _wide(4, 1, 16, 64), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)
    for c, table in ((cache, _wide(1, BIG, dtype=i32)), (_wide(BIG, 1, 16, 64), _wide(1, 4, dtype=i32)),
                     (_wide(4, 1, BIG, 64), _wide(1, 4, dtype=i32))):
        with pytest.raises(ValueError, match="int32"):
            lf.lf_paged_attention_forward(q, c, c, table, cu, kv, 1)
        with pytest.raises(ValueError, match="int32"):
            lf.lf_paged_cache_append(q, q, c, c, table, cu, kv)
    for x in (_wide(BIG, 1), _wide(1, BIG)):
        with pytest.raises(ValueError, match="int32"):
            lf.lf_layer_norm_forward(x)
        with pytest.raises(ValueError, match="int32"):
            lf.lf_layer_norm_backward(x, x, None, torch.zeros(8), torch.zeros(8))
    for call in (lambda: lf.lf_layer_norm_backward_workspace_bytes(BIG, 64),
                 lambda: lf.lf_window_attention_backward_workspace_bytes(False, 1, 1, 1, BIG, 4, 0),
                 lambda: lf.lf_paged_attention_workspace_bytes(1, 1, 1, 1, 1, BIG, 16, 4, 0)):
        with pytest.raises(ValueError, match="int32"):
            call()


def test_layer_norm_workspace_to_the_last_row_count():
    """At most 296 blocks (two per SM) of 2 N sums, for any number of rows."""
    top = (1 << 31) - 1
    for N in (1, 64, 513, 4096, 16384):
        full = 296 * 2 * N * 4
        for rows in (1 << 20, top - 300, *range(top - 9, top + 1)):
            assert lf.lf_layer_norm_backward_workspace_bytes(rows, N) == full, (rows, N)
    assert lf.lf_layer_norm_backward_workspace_bytes(1, 64) == 2 * 64 * 4
    assert lf.lf_layer_norm_backward_workspace_bytes(9, 64) == 2 * 2 * 64 * 4  # eight rows a block
