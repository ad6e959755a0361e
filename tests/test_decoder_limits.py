"""Limits of the decoder operators that need no GPU: how whole numbers reach
the library, sizes at the ends of their ranges, and the memory that a call
asks for."""
import ctypes
import enum
import random
import subprocess
import time

import numpy as np
import pytest
import torch

from sparse_attention_banded_b200 import build, lf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lf.lib()


SRC = r'''
#include "lf_paged_split.h"
using namespace lf;
extern "C" {
void plan(int n, int Hq, int Hkv, int T, int mq, int width, int w, int s, int* o) {
    PagedPlan p = paged_plan(n, Hq, Hkv, T, mq, width, w, s);
    o[0] = p.decode; o[1] = p.tensor; o[2] = p.chunk; o[3] = p.decode_splits; o[4] = p.per; o[5] = p.tensor_splits;
}
void slot(int n, int Hq, int Hkv, int T, int mq, int width, int w, int s, int b, int start, int t, int* o) {
    PagedPlan p = paged_plan(n, Hq, Hkv, T, mq, width, w, s);
    o[0] = p.decode_slot(b, start, t); o[1] = p.decode_tokens;
}
void sink_layout(int n, int T, int w, int s, int chunk, long long* o) {
    SinkRows r = {n, T, w, s, chunk};
    o[0] = r.rows(); o[1] = r.one() == r.by_seq() ? 0 : r.one() == r.by_start() ? 1 : 2; o[2] = r.first_chunk();
}
long long sink_row(int n, int T, int w, int s, int chunk, int b, int start, int len, int k) {
    SinkRows r = {n, T, w, s, chunk};
    return !r.any(len) ? -1 : k < 0 ? r.own(b, start) : r.chunk_row(b, start, k);
}
}
'''


@pytest.fixture(scope="module")
def P(tmp_path_factory):
    """The index arithmetic, compiled for the host."""
    d = tmp_path_factory.mktemp("limits")
    (d / "limits.cpp").write_text(SRC)
    so = str(d / "limits.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", build.CSRC, str(d / "limits.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


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


@pytest.mark.parametrize("n,T,max_q,Hq,Hkv,w,sinks", [
    (17, 4096 + 16, 4096, 32, 8, 1 << 30, 0), (16, 8192 + 15, 8192, 32, 8, 1 << 30, 0), (2, 2049, 2048, 32, 8, 1 << 30, 0),
    (8, 2401, 301, 32, 8, 1 << 30, 0), (300, 2000, 700, 8, 1, 4096, 4), (40, 40, 1, 16, 4, 1 << 30, 0),
    (3, 900, 300, 5, 1, 1 << 30, 0)])
def test_a_prompt_chunk_does_not_pay_for_single_tokens_pieces(P, n, T, max_q, Hq, Hkv, w, sinks):
    """Over a table of 131072 positions: the decode kernel's many pieces are
    rows of at most 16 / G tokens of a sequence (and T in all), the tensor
    cores' few pieces rows of all T; 260 bytes a row and head."""
    width, G = 131072, Hq // Hkv
    o = (ctypes.c_int * 6)()
    P.plan(n, Hq, Hkv, T, max_q, width, min(w, width), sinks, o)
    decode, tensor, _, pieces8, _, pieces64 = o
    rows = (decode and pieces8 > 1 and pieces8 * min(n * (16 // G), T)) + (tensor and pieces64 > 1 and pieces64 * T)
    got = lf.lf_paged_attention_workspace_bytes(n, Hq, Hkv, T, max_q, width // 16, 16, w, sinks)
    assert 260 * Hq * rows <= got < 260 * Hq * rows + 256


def test_workspace_of_a_chunk_next_to_single_tokens():
    """One chunk of 4096 tokens and 16 single ones: the decode rows' 128
    pieces are 72 MB at most, the chunk's pieces 34 MB each."""
    assert lf.lf_paged_attention_workspace_bytes(17, 32, 8, 4112, 4096, 8192, 16, 1 << 30, 0) <= 300 << 20


@pytest.mark.parametrize("n,T,G", [(5, 100, 1), (5, 100, 4), (5, 12, 4), (5, 20, 4), (1, 16, 1), (7, 9, 16), (3, 50, 5)])
def test_decode_slots_are_apart_and_inside(P, n, T, G):
    """Every token of a sequence short enough for the decode kernel has a slot
    of its own below decode_tokens."""
    lens = [(3 * b + 1) % (16 // G + 2) for b in range(n)]
    while sum(lens) > T:
        lens[lens.index(max(lens))] -= 1
    o = (ctypes.c_int * 2)()
    seen, start = set(), 0
    for b, m in enumerate(lens):
        for t in range(m if m * G <= 16 else 0):
            P.slot(n, G, 1, T, max(lens), 4096, 4096, 0, b, start, t, o)
            assert 0 <= o[0] < o[1] and o[0] not in seen and o[1] == min(T, n * (16 // G))
            seen.add(o[0])
        start += m


@pytest.mark.parametrize("n,Hkv", [(1000, 8), (50000, 1000), (116400, 1000), (162600, 1000), (232790, 1000), (2097151, 65535)])
def test_pieces_of_very_many_contexts(P, n, Hkv):
    """Many contexts of 131072 positions need no short pieces, however large
    the count of their tiles grows."""
    o = (ctypes.c_int * 6)()
    P.plan(n, Hkv, Hkv, n, 1, 131072, 131072, 0, o)
    assert o[2] == 128 and o[3] == 128


@pytest.mark.parametrize("Hq,max_q", [(17 * 1024, 1), (16 * 1024, 2)])
def test_too_many_pieces_are_refused_before_anything_runs(Hq, max_q):
    """2^20 sequences of 1024 key heads are 2^30 items for the tensor cores,
    next to the decode kernel's (second case) or alone."""
    heads = lambda: ctypes.byref(lf.Heads(0x10000, 1 << 20, 1 << 14, 64))  # noqa: E731
    p = ctypes.c_void_p(0x10000)
    call = lambda n: lf.lib().lf_paged_attention_forward(  # noqa: E731
        heads(), heads(), heads(), p, p, p, n, Hq, 1024, 1000, max_q, 64, 64, 16, 100, 0, 0.125, 1, p, 1 << 45, None, p)
    assert call(1 << 20) == 13


def _sink_rows(P, lens, starts, T, w, s, chunk):
    """Every partial row that the gradients of the sink keys use, checked to
    be used once and to lie inside; returns the rows in all."""
    ll = ctypes.c_longlong
    P.sink_row.restype = ll
    o = (ll * 3)()
    n = len(lens)
    P.sink_layout(n, T, w, s, chunk, o)
    rows, how, first = o
    seen = set()
    for b, m in enumerate(lens):
        # the chunks that hold a query past w, by enumeration
        want = sorted({i // chunk for i in range(w + 1, m)})
        assert not want or want[0] == first
        for k in [-1] + want if want else []:
            r = P.sink_row(n, T, w, s, chunk, b, starts[b], m, k)
            for key in range(min(s, m)):
                assert 0 <= r + key < rows and (r + key) not in seen, (b, m, k, key)
                seen.add(r + key)
        if not want:
            assert P.sink_row(n, T, w, s, chunk, b, starts[b], m, 0) == -1
    return rows, how


@pytest.mark.parametrize("seed", range(60))
def test_sink_partials_are_apart_and_inside(P, seed):
    r = random.Random(seed)
    lens = [r.choice([0, 1, 2, r.randint(0, 20), r.randint(0, 90), r.randint(0, 700)]) for _ in range(r.randint(1, 30))]
    w, s = r.choice([0, 1, 5, 16, 63, 64, 200]), r.choice([1, 4, 33, 70])
    chunk = r.choice([64, 128, 512])
    if seed % 2:
        T = sum(lens) + r.choice([0, 7])
        starts = [sum(lens[:b]) for b in range(len(lens))]
    else:  # padded
        L = max(lens + [1])
        T, starts = len(lens) * L, [b * L for b in range(len(lens))]
    rows, how = _sink_rows(P, lens, starts, T, w, s, chunk)
    assert rows <= 2 * min(len(lens) * s, T, T // (w + 2) * s) + T // chunk * s


def test_sink_partials_take_each_way(P):
    ways = set()
    for lens, w, s in (([300, 20], 5, 4), ([30, 2, 1] * 30, 25, 4), ([20, 1, 0, 2] * 40, 2, 33)):
        starts = [sum(lens[:b]) for b in range(len(lens))]
        ways.add(_sink_rows(P, lens, starts, sum(lens), w, s, 64)[1])
    assert ways == {0, 1, 2}


def test_workspace_of_many_short_documents():
    """4096 documents in 65536 tokens, 8 key heads, 64 sinks, window 256: no
    more than 254 of them can reach past the window, and 128 chunks of 512
    follow a first one: (2 * 254 + 128) * 64 rows of 512 bytes a head."""
    got = lf.lf_window_attention_backward_workspace_bytes(True, 4096, 8, 8, 65536, 256, 64)
    delta = 8 * 65536 * 4
    assert got <= delta + (2 * 254 + 128) * 64 * 8 * 512 + 256
    # and the usual call pays for its sinks alone
    assert lf.lf_window_attention_backward_workspace_bytes(False, 1, 12, 12, 16384, 256, 32) <= \
        12 * 16384 * 4 + (2 + 32) * 32 * 12 * 512 + 256


def test_sinks_that_hold_the_whole_sequence_need_no_partials():
    """Every key below the query's is a sink: plain causal attention."""
    size = lambda L, w, s: lf.lf_window_attention_backward_workspace_bytes(False, 2, 4, 4, L, w, s)  # noqa: E731
    for L in (2, 100, 4096):
        for s in (L - 1, L, L + 1, (1 << 31) - 1):
            assert size(L, 0, s) == size(L, L, 0) <= 2 * 4 * L * 4 + 255
    # (packed: 40000 sequences in 65536 tokens, whose product would pass 2^31)
    packed = lambda w, s: lf.lf_window_attention_backward_workspace_bytes(True, 40000, 4, 4, 65536, w, s)  # noqa: E731
    assert packed(5, 65536) == packed(65536, 100000) == packed(65536, 0) == 4 * 65536 * 4
    assert packed(5, 65534) == 0  # too large
