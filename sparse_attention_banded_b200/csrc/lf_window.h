// Internal declarations of the windowed causal attention (training and paged
// serving) and the stand-alone layer norm.
#pragma once

#include "lf_internal.h"
#include "lf_paged_split.h"
#include "lf_visible.h"

namespace lf {

// Items of one launch of the persistent kernels: an item's number plus the
// grid stays in 32 bits.
constexpr long long kMostItems = INT32_MAX / 2;

// One call, as the kernels see it.  Sequences are packed (cu != NULL: T = L
// rows in all) or padded (n_seqs x L rows, lens tokens).  w and sinks have
// been clamped to the longest possible sequence; sinks is 0 when every
// window reaches the sequence's start.
struct WindowArgs {
    lf_heads q, k, v;
    const int32_t* cu;
    const int32_t* lens;
    int n_seqs, Hq, Hkv, L, w, sinks;
    float scale;
    lf_dtype dtype;
    void* out;          // [B][L][Hq * 64]
    float* lse;         // [B][Hq][L]
    int* status;
    // backward
    const void* dout;   // [B][L][Hq * 64]
    lf_heads dq, dk, dv;
    float* delta;       // [B][Hq][L] workspace
    float* part;        // partial gradients of the sink keys, see below
    int chunk;          // tokens of one sink chunk
    int heads_group() const { return Hq / Hkv; }
    bool packed() const { return cu != nullptr; }
    // (worked out where it is needed: 48 bytes more of arguments are 0.4 us of
    // a launch)
    LF_HD SinkRows sink() const { return {n_seqs, cu ? L : n_seqs * L, w, sinks, chunk}; }
};

// Gradients of the sink keys: chunks of queries leave their sums in
//     part[kv head][row + key][dk, dv][64]
// at the rows that SinkRows gives them, and the window's own contribution
// goes there too (straight to dk and dv in sequences that have no chunk).  A
// last kernel adds them in a fixed order and rounds once.
// Chunks as long as an item of the window, which adds the fewest partials
// and starts; shorter, for two items per SM, only where the window's items
// (of 128 keys) leave SMs idle.  (Short ones everywhere: 536 us instead of
// 512 at 16384 packed tokens, 16 / 4 heads, window 1024; long ones
// everywhere: 178 us instead of 110 at 512 tokens, 2 heads, fp32.)
inline int sink_chunk(bool packed, int n_seqs, int Hkv, int L, int w) {
    const long long rows = (packed ? 1LL : n_seqs) * L * Hkv, share = (rows / 296 + 63) / 64 * 64;
    const long long most = w + 128 > 512 ? (w + 128 + 63LL) / 64 * 64 : 512;
    if (rows / 128 >= 296 || share > most) return (int)most;
    return (int)(share < 64 ? 64 : share);
}
// Floats of `part`.
inline size_t sink_part_floats(const SinkRows& r, int Hkv) { return (size_t)r.rows() * Hkv * 2 * 64; }

lf_status launch_window_forward_simt(const WindowArgs& a, cudaStream_t stream);   // fp32
lf_status launch_window_backward_simt(const WindowArgs& a, cudaStream_t stream);  // fp32
lf_status launch_window_forward_tc(const WindowArgs& a, cudaStream_t stream);   // 16-bit
lf_status launch_window_backward_tc(const WindowArgs& a, cudaStream_t stream);  // 16-bit
lf_status launch_sink_reduce(const WindowArgs& a, cudaStream_t stream);

// ---- paged cache ----
struct PagedArgs {
    lf_heads q;               // [T] packed new tokens
    lf_heads k_new, v_new;    // append only
    lf_heads k, v;            // cache: batch = page, token = slot in the page
    const int32_t* cu;        // [n_seqs + 1]
    const int32_t* kv_lens;   // [n_seqs]
    const int32_t* table;     // [n_seqs][max_pages]
    int n_seqs, Hq, Hkv, T, max_q, max_pages, num_pages, page_shift, w, sinks;
    float scale;
    lf_dtype dtype;
    void* out;                // [T][Hq * 64]
    int* status;
    int heads_group() const { return Hq / Hkv; }
};
// Where sequence b's n new tokens stand: kv keys in all (clamped to the
// table's width), the first new token at position `first`.  Returns false
// for a sequence that is not worked on (longer than max_q); `report` records
// what does not fit.
__device__ __forceinline__ bool paged_seq(const PagedArgs& a, int b, int n, int& kv, int& first, bool report) {
    const int raw = a.kv_lens[b], width = a.max_pages << a.page_shift;
    kv = iclamp(raw, 0, width);
    first = kv - n;
    if (report && (raw != kv || first < 0 || n > a.max_q)) record_status(a.status, b, LF_ERR_BAD_LENGTHS);
    return n <= a.max_q;
}

// The last sequence that starts at or before the token, by a whole warp: 32
// offsets at a time (one memory latency for up to 32 sequences, where a
// binary search takes five).
__device__ __forceinline__ int seq_of_token_warp(const int32_t* cu, int n_seqs, int token) {
    if (n_seqs > 512) return seq_of_token(cu, n_seqs, token);
    int count = 0;
    for (int b = 0; b < n_seqs; b += 32) {
        const int i = b + (threadIdx.x & 31);
        const unsigned before = __ballot_sync(0xffffffffu, i < n_seqs && cu[i] <= token);
        count += __popc(before);
        if (before != 0xffffffffu) break;
    }
    return imax(count - 1, 0);
}

// The offsets must ascend from 0 to at most L, and lengths fit; records the
// sequences whose do not (every access is clamped anyway).  Called by one
// group of `step` threads.
__device__ __forceinline__ void check_lengths(const int32_t* cu, const int32_t* lens, int n_seqs, int L, int* status,
                                              int thread, int step) {
    for (int b = thread; b < n_seqs; b += step) {
        const bool bad = cu ? (cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > L) : (lens && (lens[b] < 0 || lens[b] > L));
        if (bad) record_status(status, b, LF_ERR_BAD_LENGTHS);
    }
}
lf_status launch_paged_append(const PagedArgs& a, cudaStream_t stream);
lf_status launch_paged_forward(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream);
lf_status launch_paged_tc(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream);

// ---- layer norm ----
struct NormArgs {
    const void* x;
    const void* dy;
    long long x_stride, dy_stride;  // elements between rows
    const float* gamma;             // [N] or NULL
    const float* beta;              // [N] or NULL
    int rows, N;
    float eps;
    lf_dtype dtype;
    void* y;                        // forward output, backward dx: [rows][N]
    float* mean;                    // [rows] (may be NULL in the forward pass)
    float* rstd;
    float* dgamma;                  // [N] or NULL
    float* dbeta;
    float* part;                    // workspace, NULL when neither is wanted
};
lf_status launch_norm_forward(const NormArgs& a, cudaStream_t stream);
lf_status launch_norm_backward(const NormArgs& a, cudaStream_t stream);
size_t norm_backward_bytes(int rows, int N);

}  // namespace lf
