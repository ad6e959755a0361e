// How a paged attention call is cut into CTAs: which of the two kernels it
// needs and into how many pieces each cuts a context.  Host arithmetic on
// the bounds a caller gives (lengths live on the device), and the geometry
// both kernels and the merge agree on.
#pragma once

#include <stddef.h>

#include "lf_visible.h"

namespace lf {

// Sequences with at most this many query rows per key/value head (new tokens
// x grouped heads) go to the decode kernel, one mma.m16n8k16 tile of rows.
constexpr int kDecodeRows = 16;

struct PagedPlan {
    bool decode, tensor;  // kernels launched
    bool ahead;           // few items: two CTAs per SM, worked on ahead
    int chunk;            // decode: tiles of 8 keys per CTA
    int decode_splits;    // pieces of a context (n_seqs times that: its gridDim.x)
    int per;              // tensor cores: blocks of 64 keys per CTA
    int tensor_splits;    // pieces of a tile, at most
    // Partial rows of contexts in several pieces: normalised sums and their
    // log2-sum-exp.  The decode kernel cuts a context into far more pieces
    // than the tensor cores do, of far fewer rows, so each has its own:
    //     [decode_splits][decode_tokens * Hq] and [tensor_splits][T * Hq]
    // rows of 64, then the log2-sum-exps of both.  (One pointer: 32 bytes more
    // of arguments are 0.4 us of a launch.)
    int decode_tokens;    // tokens that the decode kernel may work on
    int decode_each;      // of one sequence; 0: counted over the batch's tokens
    float* part;
    LF_HD int splits() const { return imax(decode ? decode_splits : 1, tensor ? tensor_splits : 1); }
    // Where the decode kernel leaves the token t of sequence b, which starts at `start`.
    LF_HD int decode_slot(int b, int start, int t) const { return decode_each ? b * decode_each + t : start + t; }
    LF_HD size_t decode_rows(int Hq) const {
        return decode && decode_splits > 1 ? (size_t)decode_splits * decode_tokens * Hq : 0;
    }
    LF_HD size_t tensor_rows(int T, int Hq) const {
        return tensor && tensor_splits > 1 ? (size_t)tensor_splits * T * Hq : 0;
    }
    LF_HD size_t rows(int T, int Hq) const { return decode_rows(Hq) + tensor_rows(T, Hq); }
    LF_HD float* decode_o() const { return part; }
    LF_HD float* o(int Hq) const { return part + decode_rows(Hq) * 64; }
    LF_HD float* decode_lse(int T, int Hq) const { return part + rows(T, Hq) * 64; }
    LF_HD float* lse(int T, int Hq) const { return decode_lse(T, Hq) + decode_rows(Hq); }
    // Items of the tensor-core kernel.
    long long tensor_items(int T, int n_seqs, int Hkv, int G) const {
        return tensor ? (long long)packed_slots(T, n_seqs, 128 / G) * Hkv * tensor_splits : 0;
    }
};

// The tiles of 8 keys a sequence's n new tokens from position `first` see.
LF_HD KeyBlocks decode_tiles(int first, int n, int kv, int w, int sinks) {
    KeyBlocks k = {0, 0, 0};
    return first + n - 1 >= 0 ? key_blocks(first, first + n - 1, kv, w, sinks, 8) : k;
}
// The blocks of 64 keys that the tokens [t0, t1) see.
LF_HD KeyBlocks tile_key_blocks(int first, int t0, int t1, int kv, int w, int sinks) {
    KeyBlocks k = {0, 0, 0};
    return t0 < t1 && first + t1 - 1 >= 0 ? key_blocks(first + t0, first + t1 - 1, kv, w, sinks, 64) : k;
}

// Blocks of bk keys that up to max_q consecutive tokens see, at most: their
// windows span w + max_q keys.
inline long long most_blocks(int max_q, int width, int w, int sinks, int bk) {
    const long long window = ((long long)w + max_q) / bk + 2 + (sinks + (long long)bk - 1) / bk;
    const long long all = ((long long)width + bk - 1) / bk;
    return window < all ? window : all;
}

// Items of the tensor-core forward up to which each is worked on ahead, two
// CTAs per SM; more run four per SM.  Both ways, 8 heads, window 2048: 128
// items 29 and 39 us, 256 39 and 47, 320 41 and 54, 448 68 and 64, 2048 237
// and 210; window 128: 256 12.4 and 14.4, 320 18.0 and 17.2, 2048 57 and 51.
// One count for all windows: with long ones the crossing lies higher, and
// between 296 and some 400 items the other way would be up to a quarter
// faster.
constexpr int kAheadItems = 2 * 148;

// w and sinks clamped to the table's width.
inline PagedPlan paged_plan(int n_seqs, int Hq, int Hkv, int T, int max_q, int width, int w, int sinks) {
    PagedPlan p = {};
    const int G = Hq / Hkv;
    p.tensor = (long long)max_q * G > kDecodeRows;
    // (with n_seqs * max_q tokens every sequence has max_q)
    p.decode = G <= kDecodeRows && !(p.tensor && (long long)n_seqs * max_q == T);
    if (p.decode) {
        // at most kDecodeRows / G tokens of each sequence, and T in all
        const int each = kDecodeRows / G;
        p.decode_each = (long long)n_seqs * each < T ? each : 0;
        p.decode_tokens = p.decode_each ? n_seqs * each : T;
        // About two rounds of CTAs (three of 4 warps fit an SM) over the
        // widest contexts, 128 to 1024 keys each: fewer, and a warp has no
        // second step to load under its first; more, and ragged contexts
        // leave SMs idle.
        const long long tiles = most_blocks(max_q, width, w, sinks, 8), all = tiles * n_seqs * Hkv;
        const long long share = all / (2 * 3 * 148);
        p.chunk = share > 112 ? 128 : imax(((int)share + 15) / 16 * 16, 16);
        if (tiles > 1024LL * p.chunk) p.chunk = (int)((tiles + 1023) / 1024);  // at most 1024 pieces
        p.decode_splits = (int)((tiles + p.chunk - 1) / p.chunk);
    }
    if (p.tensor) {
        // In units of 0.1 us: up to 296 items run at once (two per SM, worked
        // on ahead), a block in 8 (128 items of 34 blocks: 29 us); of more,
        // 592 run at a time (four per SM), a block in 22 (measured 17, 2048
        // items of 18 blocks 135 us and of 66 471; 22 keeps to one wave more
        // readily: of calls that differ, 48 us against 52 with 16, 92 and
        // 101, 165 and 178, 82 and 75).  Pieces are joined by a further
        // kernel, worth 80 (8 us for 32768 rows of two pieces; 10 when it
        // runs anyway, for the decode kernel).
        // The device alone knows which sequences are single tokens, no tiles
        // of their own: a quarter are taken to end in a tile.  With none, a
        // quarter and all of them (us; 16 / 4 heads, contexts to 8000): 16
        // mixed lengths window 1024 29, 28, 32; 512 tokens and 64 single ones
        // window 1024 43, 45, 53, no window 110, 124, 126; 32 chunks of 33
        // and 32 single ones 47, 43, 53 and 199, 165, 174.  Pieces against
        // none, one chunk alone: 1024 tokens of 16384 144 and 209, 128 of
        // 30000 48 and 373.
        const int join = p.decode && p.decode_splits > 1 ? 10 : 80;
        const long long blocks = most_blocks(max_q, width, w, sinks, 64);
        const long long tiles = ((long long)T / (128 / G) + (p.decode ? (n_seqs + 3) / 4 : n_seqs)) * Hkv;
        long long best = -1;
        for (int s = 1; s <= 64 && (s == 1 || blocks / s >= 4); ++s) {
            const long long per = (blocks + s - 1) / s, items = tiles * s;
            const long long cost =
                (items <= kAheadItems ? (per + 2) * 8 : (items + 591) / 592 * (per + 2) * 22) + (s > 1 ? join : 0);
            if (best < 0 || cost < best) {
                best = cost;
                p.per = (int)per;
                p.tensor_splits = (int)((blocks + per - 1) / per);
                p.ahead = items <= kAheadItems;
            }
        }
    }
    return p;
}

}  // namespace lf
