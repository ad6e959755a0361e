"""The index arithmetic of the windowed attention (csrc/lf_visible.h),
compiled for the host and checked against enumeration: tiles cover every
token once, key blocks cover every visible key, masks equal the definition,
and no table or offset content leads outside its buffer."""
import ctypes
import os
import random
import subprocess

import pytest

from sparse_attention_banded_b200 import build

SRC = r'''
#include "lf_paged_split.h"
using namespace lf;
extern "C" {
int slots(int packed, int n, int L, int unit) { return token_slots(packed != 0, n, L, unit); }
void tile(const int* cu, const int* lens, int n, int L, int unit, int slot, int* o) {
    TokenTile t = token_tile(cu, lens, n, L, unit, slot);
    o[0] = t.b; o[1] = t.batch; o[2] = t.start; o[3] = t.n; o[4] = t.t0; o[5] = t.rows;
}
int token_seq(const int* cu, int n, int tok) { return seq_of_token(cu, n, tok); }
void blocks(int i0, int i1, int nk, int w, int s, int bk, int* o) {
    KeyBlocks k = key_blocks(i0, i1, nk, w, s, bk);
    o[0] = k.n;
    for (int i = 0; i < k.n && i < 4000; ++i) o[1 + i] = key_block(k, i);
}
int full(int i0, int i1, int j0, int bk, int nk, int w, int s) { return block_full(i0, i1, j0, bk, nk, w, s); }
int range_vis(int i0, int i1, int j0, int j1, int w, int s) { return range_visible(i0, i1, j0, j1, w, s); }
unsigned long long low64(int n) { return low_bits64(n); }
unsigned bits32(int i, int c0, int nk, int w, int s) { return visible_bits32(i, c0, nk, w, s); }
void plan(int n, int Hq, int Hkv, int T, int mq, int width, int w, int s, int* o) {
    PagedPlan p = paged_plan(n, Hq, Hkv, T, mq, width, w, s);
    o[0] = p.decode; o[1] = p.tensor; o[2] = p.chunk; o[3] = p.decode_splits; o[4] = p.per; o[5] = p.tensor_splits;
}
int tiles8(int first, int n, int kv, int w, int s) { return decode_tiles(first, n, kv, w, s).n; }
int blocks64(int first, int t0, int t1, int kv, int w, int s) { return tile_key_blocks(first, t0, t1, kv, w, s).n; }
int page(const int* row, int mp, int np, int sh, int j) { return page_of(row, mp, np, sh, j); }
}
'''


@pytest.fixture(scope="module")
def P(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SRC)
    so = str(d / "plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", build.CSRC, str(d / "plan.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.low64.restype, L.bits32.restype = ctypes.c_ulonglong, ctypes.c_uint
    return L


def _arr(x):
    return (ctypes.c_int * max(len(x), 1))(*x)


def _tile(P, cu, lens, n, L, unit, slot):
    o = (ctypes.c_int * 6)()
    P.tile(_arr(cu) if cu is not None else None, _arr(lens) if lens is not None else None, n, L, unit, slot, o)
    return list(o)


def _sees(i, j, w, s):
    return 0 <= j <= i and (i - j <= w or j < s)


@pytest.mark.parametrize("seed", range(20))
def test_packed_tiles_cover_each_token_once(P, seed):
    r = random.Random(seed)
    lens = [r.choice([0, 0, 1, 2, 63, 64, 65, r.randint(0, 300)]) for _ in range(r.randint(1, 12))]
    T = sum(lens) + r.choice([0, 5])
    cu = [sum(lens[:b]) for b in range(len(lens) + 1)]
    unit = r.choice([1, 2, 21, 32, 42, 64, 128])
    seen = set()
    for slot in range(P.slots(1, len(lens), T, unit)):
        b, batch, start, n, t0, rows = _tile(P, cu, None, len(lens), T, unit, slot)
        assert (batch, start, n, rows) == (0, cu[b], lens[b], lens[b])
        for t in range(t0, min(t0 + unit, n)):
            assert (b, t) not in seen
            seen.add((b, t))
    assert seen == {(b, t) for b, n in enumerate(lens) for t in range(n)}
    for tok in range(cu[-1]):
        b = P.token_seq(_arr(cu), len(lens), tok)
        assert cu[b] <= tok < cu[b + 1]


def test_padded_tiles(P):
    lens, L, unit = [0, 7, 100], 100, 32
    got = [_tile(P, None, lens, 3, L, unit, s) for s in range(P.slots(0, 3, L, unit))]
    assert len(got) == 12
    for b in range(3):
        for t in range(4):
            assert got[4 * b + t] == [b, b, 0, lens[b], 32 * t, L]
    assert _tile(P, None, [1 << 30], 1, L, unit, 0)[3] == L and _tile(P, None, [-5], 1, L, unit, 0)[3] == 0


@pytest.mark.parametrize("seed", range(30))
def test_any_offsets_stay_inside(P, seed):
    """Offsets of any content never lead to rows outside [0, T)."""
    r = random.Random(seed)
    n, T, unit = r.randint(1, 8), r.randint(1, 500), r.choice([1, 32, 64])
    cu = [r.choice([r.randint(-10, T + 10), 2 ** 31 - 1, -2 ** 31]) for _ in range(n + 1)]
    for slot in range(P.slots(1, n, T, unit)):
        b, _, start, m, t0, rows = _tile(P, cu, None, n, T, unit, slot)
        assert 0 <= b < n and 0 <= start <= T and 0 <= m and start + m <= T and t0 >= 0 and rows == m


@pytest.mark.parametrize("seed", range(40))
def test_key_blocks_and_masks(P, seed):
    r = random.Random(seed)
    nk = r.choice([1, 5, 64, 65, 200, r.randint(1, 700)])
    i0 = r.randint(0, nk - 1)
    i1 = min(nk - 1, i0 + r.choice([0, 1, 31, 63, 127]))
    w = r.choice([0, 1, 31, 63, 64, 65, r.randint(0, 700), 1 << 30])
    s = r.choice([0, 1, 4, 64, 65, 130])
    bk = r.choice([64, 128])
    o = (ctypes.c_int * 4001)()
    P.blocks(i0, i1, nk, w, s, bk, o)
    blk = list(o[1:1 + o[0]])
    assert blk == sorted(set(blk))
    need = {j // bk for i in range(i0, i1 + 1) for j in range(nk) if _sees(i, j, w, s)}
    assert need <= set(blk)
    # the only blocks without a visible key would lie between window and sinks: none are visited
    assert all(b * bk < nk for b in blk)
    for b in range((nk + bk - 1) // bk):
        keys = range(b * bk, b * bk + bk)
        full = all(j < nk and _sees(i, j, w, s) for i in range(i0, i1 + 1) for j in keys)
        assert (not P.full(i0, i1, b * bk, bk, nk, w, s)) or full
        some = any(_sees(i, j, w, s) for i in range(i0, i1 + 1) for j in keys)
        assert bool(P.range_vis(i0, i1, b * bk, b * bk + bk - 1, w, s)) or not some
    for i in {i0, i1}:
        for c0 in range(0, nk, 64):
            want = sum(1 << t for t in range(64) if c0 + t < nk and _sees(i, c0 + t, w, s))
            assert P.bits32(i, c0, nk, w, s) == want & 0xffffffff and P.bits32(i, c0 + 32, nk, w, s) == want >> 32
            assert P.bits32(-1, c0, nk, w, s) == 0


def test_low_bits(P):
    assert [P.low64(n) for n in (-5, 0, 1, 63, 64, 70)] == [0, 0, 1, 2 ** 63 - 1, 2 ** 64 - 1, 2 ** 64 - 1]


def test_pages_outside_the_table_are_missing(P):
    row = _arr([3, -1, 7, 99, 0])
    assert [P.page(row, 5, 8, 4, j) for j in (0, 15, 16, 32, 48, 64, 79, 80, -1, 2 ** 31 - 1)] == \
        [3, 3, -1, 7, -1, 0, 0, -1, -1, -1]


@pytest.mark.parametrize("seed", range(60))
def test_a_plan_covers_every_context(P, seed):
    """The pieces a call is cut into hold every block its sequences can see,
    and every sequence belongs to a kernel that is launched."""
    r = random.Random(seed)
    Hkv = r.choice([1, 2, 5])
    G = r.choice([1, 2, 3, 8, 17, 64])
    n = r.randint(1, 20)
    page = r.choice([8, 16, 64, 512])
    width = page * r.randint(1, 400)
    qs = [r.choice([0, 1, 1, r.randint(1, min(width, 300))]) for _ in range(n)]
    mq = max(max(qs), 1)
    T = max(sum(qs), 1)
    w = min(width, r.choice([0, 1, 63, 64, 100, 1000, 1 << 20]))
    s = min(width, r.choice([0, 1, 4, 64, 70]))
    o = (ctypes.c_int * 6)()
    P.plan(n, G * Hkv, Hkv, T, mq, width, w, s, o)
    decode, tensor, chunk, splits8, per, splits64 = o
    for q in qs:
        if not q:
            continue
        kv = r.randint(q, width)
        if decode and q * G <= 16:
            assert P.tiles8(kv - q, q, kv, w, s) <= chunk * splits8
        else:
            assert tensor
            TQ = 128 // G
            for t0 in range(0, q, TQ):
                assert P.blocks64(kv - q, t0, min(t0 + TQ, q), kv, w, s) <= per * splits64
