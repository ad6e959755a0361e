// C ABI entry points of the windowed causal attention, its paged form and
// the layer norm: argument validation and dispatch.
#include <limits.h>
#include <math.h>

#include "lf_window.h"

namespace lf {
namespace {

constexpr long long kInt31 = 1LL << 31;
constexpr long long kMostPositions = 1LL << 30;  // sums of two positions stay in 32 bits

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

bool known_dtype(lf_dtype t) { return t == LF_F32 || t == LF_F16 || t == LF_BF16; }

// Checks a view and copies it with usable strides for the dimensions of
// size 1 (theirs are not read).
lf_status check_view(const lf_heads* in, lf_heads* v, int batches, int heads, int tokens, lf_dtype dtype) {
    *v = *in;
    if (batches == 1) v->batch_stride = 64;
    if (heads == 1) v->head_stride = 64;
    if (tokens == 1) v->token_stride = 64;
    if (v->batch_stride <= 0 || v->head_stride <= 0 || v->token_stride <= 0) return LF_ERR_BAD_DIM;
    const int per = dtype == LF_F32 ? 4 : 8;  // 16 bytes
    if (!aligned16(v->data) || v->batch_stride % per || v->head_stride % per || v->token_stride % per)
        return LF_ERR_MISALIGNED;
    // the tensor maps of the 16-bit kernels hold strides below 2^40 bytes
    const long long most = (1LL << 40) / 4;
    if (v->batch_stride >= most || v->head_stride >= most || v->token_stride >= most) return LF_ERR_TOO_LARGE;
    return LF_OK;
}

// w and sinks clamped to sequences of at most L tokens, with the same keys
// visible: a full window holds every sink, and L - 1 sinks hold every key
// below the last.
struct Visible {
    int w, sinks;
};
Visible clamp_visible(int L, int w, int sinks) {
    const int last = imax(L - 1, 0);
    return w >= last || sinks >= last ? Visible{last, 0} : Visible{w, sinks};
}

lf_status check_window_sizes(int packed, int n_seqs, int Hq, int Hkv, int L, int w, int sinks) {
    if (n_seqs <= 0 || Hq <= 0 || Hkv <= 0 || L < 0 || w < 0 || sinks < 0) return LF_ERR_BAD_DIM;
    if (Hq % Hkv != 0 || Hq / Hkv > 64) return LF_ERR_BAD_DIM;
    const long long batches = packed ? 1 : n_seqs;
    if (batches * Hq >= kInt31 || (L > 0 && batches * Hq > (kInt31 - 1) / L)) return LF_ERR_TOO_LARGE;
    if (L >= kMostPositions) return LF_ERR_TOO_LARGE;
    if (n_seqs >= (1 << 23) || Hkv > 65535) return LF_ERR_TOO_LARGE;
    if ((long long)n_seqs * clamp_visible(L, w, sinks).sinks >= kInt31) return LF_ERR_TOO_LARGE;
    return LF_OK;
}

// The arguments both directions share.
lf_status window_args(const lf_heads* q, const lf_heads* k, const lf_heads* v, const int32_t* cu,
                      const int32_t* lens, int n_seqs, int Hq, int Hkv, int L, int w, int sinks, float scale,
                      lf_dtype dtype, WindowArgs* a) {
    if (cu && lens) return LF_ERR_BAD_DIM;
    lf_status st = check_window_sizes(cu != nullptr, n_seqs, Hq, Hkv, L, w, sinks);
    if (st != LF_OK) return st;
    if (!(scale > 0.f) || !isfinite(scale)) return LF_ERR_BAD_DIM;
    if (!known_dtype(dtype)) return LF_ERR_DTYPE;
    const int B = cu ? 1 : n_seqs;
    if ((st = check_view(q, &a->q, B, Hq, L, dtype)) != LF_OK) return st;
    if ((st = check_view(k, &a->k, B, Hkv, L, dtype)) != LF_OK) return st;
    if ((st = check_view(v, &a->v, B, Hkv, L, dtype)) != LF_OK) return st;
    if ((reinterpret_cast<uintptr_t>(cu) | reinterpret_cast<uintptr_t>(lens)) & 3) return LF_ERR_MISALIGNED;
    a->cu = cu;
    a->lens = lens;
    a->n_seqs = n_seqs;
    a->Hq = Hq;
    a->Hkv = Hkv;
    a->L = L;
    const Visible vis = clamp_visible(L, w, sinks);
    a->w = vis.w;
    a->sinks = vis.sinks;
    a->chunk = sink_chunk(cu != nullptr, n_seqs, Hkv, L, a->w);
    a->scale = scale;
    a->dtype = dtype;
    return LF_OK;
}

lf_status check_paged_sizes(int n_seqs, int Hq, int Hkv, int T, int max_pages, int num_pages, int page_size) {
    if (n_seqs <= 0 || Hq <= 0 || Hkv <= 0 || T < 0 || max_pages <= 0 || num_pages <= 0) return LF_ERR_BAD_DIM;
    if (page_size < 8 || page_size > 4096 || (page_size & (page_size - 1))) return LF_ERR_BAD_DIM;
    if (Hq % Hkv != 0 || Hq / Hkv > 64) return LF_ERR_BAD_DIM;
    if ((T > 0 && Hq > (kInt31 - 1) / T) || (long long)max_pages * page_size > (1LL << 24) || n_seqs >= (1 << 21) ||
        Hkv > 65535)
        return LF_ERR_TOO_LARGE;
    return LF_OK;
}

int log2_of(int n) {
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

lf_status check_cache(const lf_heads* k, const lf_heads* v, int num_pages, int Hkv, int page_size, lf_dtype dtype,
                      PagedArgs* a) {
    lf_status st = check_view(k, &a->k, num_pages, Hkv, page_size, dtype);
    return st != LF_OK ? st : check_view(v, &a->v, num_pages, Hkv, page_size, dtype);
}

bool misaligned4(const void* a, const void* b, const void* c) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c)) & 3) != 0;
}

lf_status check_norm(int rows, int N, long long stride, long long stride2, lf_dtype dtype) {
    if (rows < 0 || N <= 0 || stride < N || stride2 < N) return LF_ERR_BAD_DIM;
    if (N > 16384) return LF_ERR_TOO_LARGE;
    return known_dtype(dtype) ? LF_OK : LF_ERR_DTYPE;
}

}  // namespace
}  // namespace lf

using namespace lf;

extern "C" {

lf_status lf_window_attention_forward(const lf_heads* q, const lf_heads* k, const lf_heads* v,
                                      const int32_t* cu_seqlens, const int32_t* seq_lens, int n_seqs, int Hq,
                                      int Hkv, int L, int w, int sinks, float scale, lf_dtype dtype,
                                      lf_stream_t stream, void* out, float* lse) {
    if (!q || !k || !v) return LF_ERR_NULL;
    if (L != 0 && (!q->data || !k->data || !v->data || !out || !lse)) return LF_ERR_NULL;
    WindowArgs a = {};
    lf_status st = window_args(q, k, v, cu_seqlens, seq_lens, n_seqs, Hq, Hkv, L, w, sinks, scale, dtype, &a);
    if (st != LF_OK) return st;
    if (!aligned16(out) || !aligned16(lse)) return LF_ERR_MISALIGNED;
    if (L == 0) return LF_OK;
    DeviceCtx* d = current_device(&st);
    if (!d) return st;
    a.out = out;
    a.lse = lse;
    a.status = d->status;
    return dtype == LF_F32 ? launch_window_forward_simt(a, (cudaStream_t)stream)
                           : launch_window_forward_tc(a, (cudaStream_t)stream);
}

size_t lf_window_attention_backward_workspace_bytes(int packed, int n_seqs, int Hq, int Hkv, int L, int w, int sinks) {
    if (check_window_sizes(packed, n_seqs, Hq, Hkv, L, w, sinks) != LF_OK || L == 0) return 0;
    size_t n = align256((size_t)(packed ? 1 : n_seqs) * Hq * L * sizeof(float));  // delta
    const Visible vis = clamp_visible(L, w, sinks);
    if (vis.sinks > 0) {
        const SinkRows r = {n_seqs, packed ? L : n_seqs * L, vis.w, vis.sinks,
                            sink_chunk(packed != 0, n_seqs, Hkv, L, vis.w)};
        n += align256(sink_part_floats(r, Hkv) * sizeof(float));
    }
    return n;
}

lf_status lf_window_attention_backward(const lf_heads* q, const lf_heads* k, const lf_heads* v, const void* out,
                                       const float* lse, const void* dout, const int32_t* cu_seqlens,
                                       const int32_t* seq_lens, int n_seqs, int Hq, int Hkv, int L, int w, int sinks,
                                       float scale, lf_dtype dtype, void* workspace, size_t workspace_bytes,
                                       lf_stream_t stream, const lf_heads* dq, const lf_heads* dk,
                                       const lf_heads* dv) {
    if (!q || !k || !v || !dq || !dk || !dv) return LF_ERR_NULL;
    if (L != 0 && (!q->data || !k->data || !v->data || !dq->data || !dk->data || !dv->data || !out || !lse || !dout))
        return LF_ERR_NULL;
    WindowArgs a = {};
    lf_status st = window_args(q, k, v, cu_seqlens, seq_lens, n_seqs, Hq, Hkv, L, w, sinks, scale, dtype, &a);
    if (st != LF_OK) return st;
    const int B = cu_seqlens ? 1 : n_seqs;
    if ((st = check_view(dq, &a.dq, B, Hq, L, dtype)) != LF_OK) return st;
    if ((st = check_view(dk, &a.dk, B, Hkv, L, dtype)) != LF_OK) return st;
    if ((st = check_view(dv, &a.dv, B, Hkv, L, dtype)) != LF_OK) return st;
    if (!aligned16(out) || !aligned16(lse) || !aligned16(dout)) return LF_ERR_MISALIGNED;
    if (L == 0) return LF_OK;
    const size_t need =
        lf_window_attention_backward_workspace_bytes(cu_seqlens != nullptr, n_seqs, Hq, Hkv, L, w, sinks);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need)
        return LF_ERR_WORKSPACE;
    DeviceCtx* d = current_device(&st);
    if (!d) return st;
    a.out = const_cast<void*>(out);
    a.lse = const_cast<float*>(lse);
    a.dout = dout;
    a.delta = static_cast<float*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256((size_t)B * Hq * L * sizeof(float)));
    a.status = d->status;
    return dtype == LF_F32 ? launch_window_backward_simt(a, (cudaStream_t)stream)
                           : launch_window_backward_tc(a, (cudaStream_t)stream);
}

lf_status lf_paged_cache_append(const lf_heads* k_new, const lf_heads* v_new, const lf_heads* k_cache,
                                const lf_heads* v_cache, const int32_t* block_table, const int32_t* cu_seqlens,
                                const int32_t* kv_lens, int n_seqs, int Hkv, int T, int max_pages, int num_pages,
                                int page_size, lf_dtype dtype, lf_stream_t stream) {
    if (!k_new || !v_new || !k_cache || !v_cache) return LF_ERR_NULL;
    if (T != 0 && (!k_new->data || !v_new->data || !k_cache->data || !v_cache->data || !block_table || !cu_seqlens ||
                   !kv_lens))
        return LF_ERR_NULL;
    PagedArgs a = {};
    lf_status st = check_paged_sizes(n_seqs, Hkv, Hkv, T, max_pages, num_pages, page_size);
    if (st != LF_OK) return st;
    if (dtype != LF_F16 && dtype != LF_BF16) return LF_ERR_DTYPE;
    if ((st = check_view(k_new, &a.k_new, 1, Hkv, T, dtype)) != LF_OK) return st;
    if ((st = check_view(v_new, &a.v_new, 1, Hkv, T, dtype)) != LF_OK) return st;
    if ((st = check_cache(k_cache, v_cache, num_pages, Hkv, page_size, dtype, &a)) != LF_OK) return st;
    if (misaligned4(block_table, cu_seqlens, kv_lens)) return LF_ERR_MISALIGNED;
    if (T == 0) return LF_OK;
    DeviceCtx* d = current_device(&st);
    if (!d) return st;
    a.cu = cu_seqlens;
    a.kv_lens = kv_lens;
    a.table = block_table;
    a.n_seqs = n_seqs;
    a.Hq = a.Hkv = Hkv;
    a.T = T;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_shift = log2_of(page_size);
    a.status = d->status;
    return launch_paged_append(a, (cudaStream_t)stream);
}

size_t lf_paged_attention_workspace_bytes(int n_seqs, int Hq, int Hkv, int T, int max_q_len, int max_pages,
                                          int page_size, int w, int sinks) {
    if (check_paged_sizes(n_seqs, Hq, Hkv, T, max_pages, 1, page_size) != LF_OK || T == 0 || max_q_len <= 0 || w < 0 ||
        sinks < 0)
        return 0;
    const int width = max_pages * page_size;
    const PagedPlan p =
        paged_plan(n_seqs, Hq, Hkv, T, imin(max_q_len, T), width, imin(w, width), imin(sinks, width));
    const size_t rows = p.rows(T, Hq);
    return rows * 64 * sizeof(float) + align256(rows * sizeof(float));
}

lf_status lf_paged_attention_forward(const lf_heads* q, const lf_heads* k_cache, const lf_heads* v_cache,
                                     const int32_t* block_table, const int32_t* cu_seqlens, const int32_t* kv_lens,
                                     int n_seqs, int Hq, int Hkv, int T, int max_q_len, int max_pages, int num_pages,
                                     int page_size, int w, int sinks, float scale, lf_dtype dtype, void* workspace,
                                     size_t workspace_bytes, lf_stream_t stream, void* out) {
    if (!q || !k_cache || !v_cache) return LF_ERR_NULL;
    if (T != 0 && (!q->data || !k_cache->data || !v_cache->data || !block_table || !cu_seqlens || !kv_lens || !out))
        return LF_ERR_NULL;
    PagedArgs a = {};
    lf_status st = check_paged_sizes(n_seqs, Hq, Hkv, T, max_pages, num_pages, page_size);
    if (st != LF_OK) return st;
    if (max_q_len < 0 || (T > 0 && max_q_len == 0) || w < 0 || sinks < 0 || !(scale > 0.f) || !isfinite(scale))
        return LF_ERR_BAD_DIM;
    if (dtype != LF_F16 && dtype != LF_BF16) return LF_ERR_DTYPE;
    if ((st = check_view(q, &a.q, 1, Hq, T, dtype)) != LF_OK) return st;
    if ((st = check_cache(k_cache, v_cache, num_pages, Hkv, page_size, dtype, &a)) != LF_OK) return st;
    if (!aligned16(out) || misaligned4(block_table, cu_seqlens, kv_lens)) return LF_ERR_MISALIGNED;
    if (T == 0) return LF_OK;
    const size_t need =
        lf_paged_attention_workspace_bytes(n_seqs, Hq, Hkv, T, max_q_len, max_pages, page_size, w, sinks);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need))
        return LF_ERR_WORKSPACE;
    // (before the first launch: a refused call does nothing)
    const int width = max_pages * page_size, G = Hq / Hkv;
    PagedPlan plan =
        paged_plan(n_seqs, Hq, Hkv, T, imin(max_q_len, T), width, imin(w, width), imin(sinks, width));
    if (plan.decode && (long long)n_seqs * plan.decode_splits >= kInt31) return LF_ERR_TOO_LARGE;
    if (plan.tensor_items(T, n_seqs, Hkv, G) > kMostItems) return LF_ERR_TOO_LARGE;
    DeviceCtx* d = current_device(&st);
    if (!d) return st;
    a.cu = cu_seqlens;
    a.kv_lens = kv_lens;
    a.table = block_table;
    a.n_seqs = n_seqs;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.T = T;
    a.max_q = imin(max_q_len, T);
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_shift = log2_of(page_size);
    a.w = imin(w, width);
    a.sinks = imin(sinks, width);
    a.scale = scale;
    a.dtype = dtype;
    a.out = out;
    a.status = d->status;
    plan.part = static_cast<float*>(workspace);
    return launch_paged_forward(a, plan, (cudaStream_t)stream);
}

lf_status lf_layer_norm_forward(const void* x, long long x_stride, const float* gamma, const float* beta, int rows,
                                int N, float eps, lf_dtype dtype, lf_stream_t stream, void* y, float* mean,
                                float* rstd) {
    if (rows != 0 && (!x || !y)) return LF_ERR_NULL;
    lf_status st = check_norm(rows, N, x_stride, N, dtype);
    if (st != LF_OK) return st;
    if (!(eps >= 0.f) || !isfinite(eps)) return LF_ERR_BAD_DIM;
    for (const void* p : {x, (const void*)gamma, (const void*)beta, (const void*)y})
        if (!aligned16(p)) return LF_ERR_MISALIGNED;
    if (misaligned4(mean, rstd, nullptr)) return LF_ERR_MISALIGNED;
    if (rows == 0) return LF_OK;
    if (!current_device(&st)) return st;
    NormArgs a = {};
    a.x = x;
    a.x_stride = x_stride;
    a.gamma = gamma;
    a.beta = beta;
    a.rows = rows;
    a.N = N;
    a.eps = eps;
    a.dtype = dtype;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    return launch_norm_forward(a, (cudaStream_t)stream);
}

size_t lf_layer_norm_backward_workspace_bytes(int rows, int N) {
    if (rows <= 0 || N <= 0 || N > 16384) return 0;
    return norm_backward_bytes(rows, N);
}

lf_status lf_layer_norm_backward(const void* dy, long long dy_stride, const void* x, long long x_stride,
                                 const float* gamma, const float* mean, const float* rstd, int rows, int N,
                                 lf_dtype dtype, void* workspace, size_t workspace_bytes, lf_stream_t stream,
                                 void* dx, float* dgamma, float* dbeta) {
    if (rows != 0 && (!dy || !x || !mean || !rstd || !dx)) return LF_ERR_NULL;
    lf_status st = check_norm(rows, N, x_stride, dy_stride, dtype);
    if (st != LF_OK) return st;
    for (const void* p : {dy, x, (const void*)gamma, (const void*)dx, (const void*)dgamma, (const void*)dbeta})
        if (!aligned16(p)) return LF_ERR_MISALIGNED;
    if (misaligned4(mean, rstd, nullptr)) return LF_ERR_MISALIGNED;
    const bool params = dgamma || dbeta;
    if (params && rows > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
                               workspace_bytes < norm_backward_bytes(rows, N)))
        return LF_ERR_WORKSPACE;
    if (rows == 0 && !params) return LF_OK;
    if (!current_device(&st)) return st;
    if (rows == 0) {
        for (float* p : {dgamma, dbeta})
            if (p && cudaMemsetAsync(p, 0, (size_t)N * sizeof(float), (cudaStream_t)stream) != cudaSuccess)
                return LF_ERR_CUDA;
        return LF_OK;
    }
    NormArgs a = {};
    a.x = x;
    a.dy = dy;
    a.x_stride = x_stride;
    a.dy_stride = dy_stride;
    a.gamma = gamma;
    a.rows = rows;
    a.N = N;
    a.dtype = dtype;
    a.y = dx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.part = params ? static_cast<float*>(workspace) : nullptr;
    return launch_norm_backward(a, (cudaStream_t)stream);
}

}  // extern "C"
