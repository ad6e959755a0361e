// Index arithmetic of the windowed causal attention with sinks: which
// sequence a tile belongs to, which keys a query sees, which key blocks a
// tile of queries visits.  Plain integer code, compiled for the device by
// the kernels and for the host by the tests.
//
// A query at position i of its sequence sees the keys
//     { j <= i : i - j <= w or j < sinks }.
// The entry points clamp w and sinks to the longest sequence, so that sums
// and differences of positions, w and block offsets stay in 32 bits.
#pragma once

#ifdef __CUDACC__
#define LF_HD __host__ __device__ __forceinline__
#else
#define LF_HD inline
#endif

namespace lf {

LF_HD int imin(int a, int b) { return a < b ? a : b; }
LF_HD int imax(int a, int b) { return a > b ? a : b; }
LF_HD int iclamp(int x, int lo, int hi) { return imin(imax(x, lo), hi); }

LF_HD bool key_visible(int i, int j, int w, int sinks) { return j >= 0 && j <= i && (i - j <= w || j < sinks); }

// ---- packed sequences -----------------------------------------------------
// cu[0..n_seqs] are the sequences' first tokens (cu[n_seqs]: the end).  Work
// on tiles of `unit` tokens is numbered without a prefix sum over tile
// counts: sequence b owns the slots from cu[b] / unit + b on.  There are at
// least ceil(len / unit) of them before the next sequence's, because
// floor((x + n) / u) - floor(x / u) + 1 >= ceil(n / u); surplus slots have
// no tokens.  Offsets are clamped to [0, T], so no content reaches outside.
LF_HD int seq_slot(const int* cu, int b, int T, int unit) { return iclamp(cu[b], 0, T) / unit + b; }
LF_HD int packed_slots(int T, int n_seqs, int unit) { return T / unit + n_seqs; }
LF_HD int find_seq(const int* cu, int n_seqs, int T, int unit, int slot) {
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (seq_slot(cu, mid, T, unit) <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The last sequence that starts at or before the token.
LF_HD int seq_of_token(const int* cu, int n_seqs, int token) {
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (cu[mid] <= token) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// One tile of tokens: sequence b, tokens [t0, min(t0 + unit, n)) of its n.
struct TokenTile {
    int b;      // sequence
    int batch;  // batch index of its rows (0 when packed)
    int start;  // row of its first token
    int n;      // tokens of the sequence
    int t0;     // first token of the tile
    int rows;   // rows that belong to the sequence's storage (n, or L when padded)
};

// slot -> tile; cu NULL: sequences of L rows each, lens (may be NULL) tokens.
LF_HD TokenTile token_tile(const int* cu, const int* lens, int n_seqs, int L, int unit, int slot) {
    TokenTile t;
    if (cu) {
        t.b = find_seq(cu, n_seqs, L, unit, slot);
        t.batch = 0;
        t.start = iclamp(cu[t.b], 0, L);
        t.n = imax(0, iclamp(cu[t.b + 1], 0, L) - t.start);
        t.t0 = (slot - (t.start / unit + t.b)) * unit;
        t.rows = t.n;
        if (t.t0 < 0) t.t0 = t.rows;  // only with offsets that are not ascending: no work
    } else {
        const int per = (L + unit - 1) / unit;
        t.b = slot / per;
        t.batch = t.b;
        t.start = 0;
        t.n = lens ? iclamp(lens[t.b], 0, L) : L;
        t.t0 = (slot - t.b * per) * unit;
        t.rows = L;
    }
    return t;
}
LF_HD int token_slots(bool packed, int n_seqs, int L, int unit) {
    return packed ? packed_slots(L, n_seqs, unit) : n_seqs * ((L + unit - 1) / unit);
}

// ---- key blocks of a tile of queries --------------------------------------
// Queries at positions [i0, i1], keys [0, n_keys): the blocks of `bk` keys
// that hold a visible key: the blocks of the sinks before the window, then
// the window's.  The first query's own key exists (i0 < n_keys) unless there
// is no key at all.
struct KeyBlocks {
    int n_sink, lo, n;
};
LF_HD KeyBlocks key_blocks(int i0, int i1, int n_keys, int w, int sinks, int bk) {
    KeyBlocks k;
    const int last = imin(i1, n_keys - 1);
    k.n_sink = k.lo = k.n = 0;
    if (i0 < 0) i0 = 0;
    if (last < 0) return k;
    const int lo_key = imax(0, i0 - w);
    k.lo = lo_key / bk;
    k.n_sink = imin((sinks + bk - 1) / bk, k.lo);
    k.n = k.n_sink + last / bk - k.lo + 1;
    return k;
}
LF_HD int key_block(const KeyBlocks& k, int idx) { return idx < k.n_sink ? idx : k.lo + (idx - k.n_sink); }

// Is every key of [j0, j0 + bk) visible to every query of [i0, i1]?
LF_HD bool block_full(int i0, int i1, int j0, int bk, int n_keys, int w, int sinks) {
    const int j1 = j0 + bk - 1;
    return j1 < n_keys && j1 <= i0 && (i1 - j0 <= w || j1 < sinks);
}
// Does any query of [i0, i1] see a key of [j0, j1]?
LF_HD bool range_visible(int i0, int i1, int j0, int j1, int w, int sinks) {
    if (j1 > i1) j1 = i1;  // keys past the last query are seen by none
    if (j0 > j1) return false;
    return i0 - j1 <= w || j0 < sinks;
}

// Bits [0, n) of a 64-bit word, n clamped to [0, 64].
LF_HD unsigned long long low_bits64(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}
// Bits [0, n) of a 32-bit word, n clamped to [0, 32].
LF_HD unsigned low_bits32(int n) {
#ifdef __CUDA_ARCH__
    unsigned m;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(m) : "r"(imax(n, 0)));
    return m;
#else
    return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
#endif
}
// Keys c0 .. c0 + 31 that the query at position i sees, of n_keys.
LF_HD unsigned visible_bits32(int i, int c0, int n_keys, int w, int sinks) {
    return low_bits32(imin(i + 1, n_keys) - c0) & (~low_bits32(i - w - c0) | low_bits32(sinks - c0));
}

// ---- partial gradients of the sink keys -----------------------------------
// The queries that see a sink from outside its window are cut into chunks of
// `chunk` tokens of their sequence, of which those that hold only queries up
// to w are skipped.  A sequence of at most w + 1 tokens has none; of the
// others, `rows` rows a key/value head hold
//   own(b, start) + key                the window's own contribution,
//   chunk_row(b, start, k) + key       chunk k's,
// for each sink key of the sequence.  `start` counts tokens over the batch (b
// * L when padded), T in all.  No prefix sums: sequence b has the rows of
// sequence b, or, where that is less, those of start / (w + 2) (sequences
// that long are at least w + 2 apart), or those of its own tokens; its chunks
// after the first have the slots from start / chunk on, since there are at
// most n / chunk of them.
struct SinkRows {
    int n_seqs, T, w, sinks, chunk;
    LF_HD bool any(int n) const { return n > w + 1; }
    LF_HD int first_chunk() const { return (w + 1) / chunk; }
    LF_HD long long by_seq() const { return (long long)n_seqs * sinks; }
    LF_HD long long by_start() const { return (long long)(T / (w + 2)) * sinks; }
    // Rows of the windows, and of the first chunks.
    LF_HD long long one() const {
        const long long r = by_start() < by_seq() ? by_start() : by_seq();
        return T < r ? T : r;
    }
    LF_HD long long rows() const { return 2 * one() + (long long)(T / chunk) * sinks; }
    LF_HD long long own(int b, int start) const {
        const long long r = one();
        return r == by_seq() ? (long long)b * sinks : r == by_start() ? (long long)(start / (w + 2)) * sinks : start;
    }
    LF_HD long long chunk_row(int b, int start, int k) const {
        k -= first_chunk();
        return k == 0 ? one() + own(b, start) : 2 * one() + (long long)(start / chunk + k - 1) * sinks;
    }
};

// ---- paged cache ----------------------------------------------------------
// The page of key position j in a sequence's table row, -1 where the table
// has none: past its width, or an entry outside [0, num_pages).
LF_HD int page_of(const int* table_row, int max_pages, int num_pages, int page_shift, int j) {
    const int k = j >> page_shift;
    if (j < 0 || k >= max_pages) return -1;
    const int p = table_row[k];
    return p >= 0 && p < num_pages ? p : -1;
}

}  // namespace lf
