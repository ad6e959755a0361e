// Windowed causal attention with sinks in fp32 on the CUDA cores, forward and
// backward (and the last step of every dtype's sink gradients).
//
//   forward   one CTA per tile of 64 query rows (64 / G tokens times the G
//             query heads of a key/value head), online softmax over blocks
//             of 64 keys:  m' = max(m, max s), l' = l 2^(m - m') + sum 2^(s - m'),
//             O' = O 2^(m - m') + P V.
//   backward  dQ: one CTA per query tile;  dK, dV: one CTA per block of 64
//             keys, over the query tiles that see it, all G heads of the
//             group in one accumulator.  P is recomputed from the saved
//             log-sum-exp.  Each sum has one owner and one order: no atomics.
//
// The three products of a block pair run from shared memory with a 4 x 4
// register tile per thread (8 float4 loads for 64 FMAs).  Shared-memory
// bandwidth bounds them when the tiles fill the GPU; 512 tokens, 2 heads,
// window 64 (a forward and backward of 110 us) are 16 tiles a kernel, each a
// chain of a few blocks.
#include "lf_convert.cuh"
#include "lf_window.h"

namespace lf {
namespace {

constexpr int kT = 64;      // rows and keys per tile
constexpr int kD = 64;      // head dim
constexpr int kLd = 68;     // padded row of a shared tile (floats)
constexpr int kThreads = 256;
constexpr int kTile = kT * kLd;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 64 rows of 64 into a shared tile; row(r) is the row's address, NULL: zeros.
template <typename F>
__device__ __forceinline__ void load_tile(float* dst, F row) {
    const int c = (threadIdx.x & 15) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (threadIdx.x >> 4) + 16 * i;
        const float* p = row(r);
        *reinterpret_cast<float4*>(dst + r * kLd + c) =
            p ? *reinterpret_cast<const float4*>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// acc[i][j] = A[4 ty + i] . B[tx + 16 j]
__device__ __forceinline__ void tile_nt(float (&acc)[4][4], const float* A, const float* B, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < kD; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * kLd + d);
            b[i] = *reinterpret_cast<const float4*>(B + (tx + 16 * i) * kLd + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
                acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
                acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
                acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
            }
    }
}

// acc[i][0..3] += sum_k P[4 ty + i][k] V[k][4 tx ..]
__device__ __forceinline__ void tile_nn(float (&acc)[4][4], const float* P, const float* V, int ty, int tx) {
#pragma unroll 4
    for (int k = 0; k < kT; k += 4) {
        float4 p[4], v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[i] = *reinterpret_cast<const float4*>(P + (4 * ty + i) * kLd + k);
            v[i] = *reinterpret_cast<const float4*>(V + (k + i) * kLd + 4 * tx);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float pk[4] = {p[i].x, p[i].y, p[i].z, p[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][0] = fmaf(pk[j], v[j].x, acc[i][0]);
                acc[i][1] = fmaf(pk[j], v[j].y, acc[i][1]);
                acc[i][2] = fmaf(pk[j], v[j].z, acc[i][2]);
                acc[i][3] = fmaf(pk[j], v[j].w, acc[i][3]);
            }
        }
    }
}

// Sum / max over the 16 threads that share ty.
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float max16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

__device__ __forceinline__ float* view_row(const lf_heads& v, int batch, int head, int token) {
    return static_cast<float*>(v.data) + batch * v.batch_stride + head * v.head_stride + token * v.token_stride;
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// ---------------------------------------------------------------- forward
__global__ void __launch_bounds__(kThreads) forward_kernel(const __grid_constant__ WindowArgs a) {
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + kTile, *V = K + kTile, *P = V + kTile;
    const int G = a.Hq / a.Hkv, TQ = kT / G, hk = blockIdx.y;
    if (blockIdx.x == 0 && hk == 0) check_lengths(a.cu, a.lens, a.n_seqs, a.L, a.status, threadIdx.x, blockDim.x);
    const TokenTile t = token_tile(a.cu, a.lens, a.n_seqs, a.L, TQ, blockIdx.x);
    if (t.t0 >= t.rows) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    auto q_row = [&](int r) -> const float* {
        const int i = t.t0 + r / G;
        return r < TQ * G && i < t.n ? view_row(a.q, t.batch, hk * G + r % G, t.start + i) : nullptr;
    };
    load_tile(Q, q_row);
    float m[4], l[4], o[4][4];
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        pos[i] = r < TQ * G ? t.t0 + r / G : INT32_MAX;
        if (pos[i] >= t.n) pos[i] = -1;  // sees nothing
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
    }
    const float sc = a.scale * kLog2e;
    const int i1 = imin(t.t0 + TQ, t.n) - 1;
    KeyBlocks kb = {0, 0, 0};
    if (t.t0 < t.n) kb = key_blocks(t.t0, i1, t.n, a.w, a.sinks, kT);
    for (int n = 0; n < kb.n; ++n) {
        const int c0 = key_block(kb, n) * kT;
        __syncthreads();
        load_tile(K, [&](int r) -> const float* {
            return c0 + r < t.n ? view_row(a.k, t.batch, hk, t.start + c0 + r) : nullptr;
        });
        load_tile(V, [&](int r) -> const float* {
            return c0 + r < t.n ? view_row(a.v, t.batch, hk, t.start + c0 + r) : nullptr;
        });
        __syncthreads();
        float s[4][4];
        tile_nt(s, Q, K, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = c0 + tx + 16 * j;
                s[i][j] = key_visible(pos[i], key, a.w, a.sinks) && key < t.n ? s[i][j] * sc : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            const float mn = fmaxf(m[i], max16(mx));
            const float base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - base);
                sum += p;
                P[(4 * ty + i) * kLd + tx + 16 * j] = p;
            }
            m[i] = mn;
            l[i] = l[i] * f + sum16(sum);
#pragma unroll
            for (int c = 0; c < 4; ++c) o[i][c] *= f;
        }
        __syncwarp();  // a row of P is written and read by the same half warp
        tile_nn(o, P, V, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i, tok = t.t0 + r / G, h = hk * G + r % G;
        if (r >= TQ * G || tok >= t.rows) continue;
        const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][c] *= inv;
        const size_t row = (size_t)t.batch * a.L + t.start + tok;
        store4(static_cast<float*>(a.out) + (row * a.Hq + h) * kD + 4 * tx, o[i]);
        if (tx == 0)
            a.lse[((size_t)t.batch * a.Hq + h) * a.L + t.start + tok] =
                l[i] == 0.f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
    }
}

// ---------------------------------------------------------------- dQ
// Also leaves delta = rowsum(dO * out) for the kernels of dK and dV.
__global__ void __launch_bounds__(kThreads) dq_kernel(const __grid_constant__ WindowArgs a) {
    extern __shared__ float sm[];
    float *Q = sm, *dO = Q + kTile, *K = dO + kTile, *V = K + kTile, *S = V + kTile;
    const int G = a.Hq / a.Hkv, TQ = kT / G, hk = blockIdx.y;
    if (blockIdx.x == 0 && hk == 0) check_lengths(a.cu, a.lens, a.n_seqs, a.L, a.status, threadIdx.x, blockDim.x);
    const TokenTile t = token_tile(a.cu, a.lens, a.n_seqs, a.L, TQ, blockIdx.x);
    if (t.t0 >= t.rows) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    auto live = [&](int r) { return r < TQ * G && t.t0 + r / G < t.n; };
    auto o_off = [&](int r) {
        return (((size_t)t.batch * a.L + t.start + t.t0 + r / G) * a.Hq + hk * G + r % G) * kD;
    };
    load_tile(Q, [&](int r) -> const float* {
        return live(r) ? view_row(a.q, t.batch, hk * G + r % G, t.start + t.t0 + r / G) : nullptr;
    });
    load_tile(dO, [&](int r) -> const float* { return live(r) ? static_cast<const float*>(a.dout) + o_off(r) : nullptr; });
    load_tile(K, [&](int r) -> const float* { return live(r) ? static_cast<const float*>(a.out) + o_off(r) : nullptr; });
    __syncthreads();
    float delta[4], lse[4], acc[4][4];
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i, tok = t.t0 + r / G, h = hk * G + r % G;
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            s = fmaf(dO[r * kLd + 4 * tx + c], K[r * kLd + 4 * tx + c], s);
            acc[i][c] = 0.f;
        }
        delta[i] = sum16(s);
        pos[i] = live(r) ? tok : -1;
        lse[i] = 0.f;
        if (live(r)) {
            const size_t at = ((size_t)t.batch * a.Hq + h) * a.L + t.start + tok;
            lse[i] = a.lse[at] * kLog2e;
            if (tx == 0) a.delta[at] = delta[i];
        }
    }
    const float sc = a.scale * kLog2e;
    KeyBlocks kb = {0, 0, 0};
    if (t.t0 < t.n) kb = key_blocks(t.t0, imin(t.t0 + TQ, t.n) - 1, t.n, a.w, a.sinks, kT);
    for (int n = 0; n < kb.n; ++n) {
        const int c0 = key_block(kb, n) * kT;
        __syncthreads();
        load_tile(K, [&](int r) -> const float* {
            return c0 + r < t.n ? view_row(a.k, t.batch, hk, t.start + c0 + r) : nullptr;
        });
        load_tile(V, [&](int r) -> const float* {
            return c0 + r < t.n ? view_row(a.v, t.batch, hk, t.start + c0 + r) : nullptr;
        });
        __syncthreads();
        float s[4][4], dp[4][4];
        tile_nt(s, Q, K, ty, tx);
        tile_nt(dp, dO, V, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = c0 + tx + 16 * j;
                const bool vis = key_visible(pos[i], key, a.w, a.sinks) && key < t.n;
                S[(4 * ty + i) * kLd + tx + 16 * j] =
                    vis ? exp2f(fmaf(s[i][j], sc, -lse[i])) * (dp[i][j] - delta[i]) : 0.f;
            }
        __syncwarp();
        tile_nn(acc, S, K, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i, tok = t.t0 + r / G;
        if (r >= TQ * G || tok >= t.rows) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] *= a.scale;
        store4(view_row(a.dq, t.batch, hk * G + r % G, t.start + tok) + 4 * tx, acc[i]);
    }
}

// ---------------------------------------------------------------- dK, dV
// kSink false: one block of 64 keys over the queries that hold it in their
// window.  kSink true: one block of sink keys over a chunk of the queries
// that see it from outside their window; writes fp32 partial sums.  blockIdx.x
// counts `slots` tiles of keys, or of queries for each block of sink keys.
template <bool kSink>
__global__ void __launch_bounds__(kThreads) dkv_kernel(const __grid_constant__ WindowArgs a, int slots) {
    extern __shared__ float sm[];
    float *K = sm, *V = K + kTile, *Q = V + kTile, *dO = Q + kTile, *P = dO + kTile, *S = P + kTile;
    __shared__ float lse_s[kT], delta_s[kT];
    const int G = a.Hq / a.Hkv, TQ = kT / G, hk = blockIdx.y;
    const TokenTile t = token_tile(a.cu, a.lens, a.n_seqs, a.L, kSink ? a.chunk : kT, blockIdx.x % slots);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (kSink ? t.t0 >= t.n : t.t0 >= t.rows) return;
    const int n_sink = a.sink().any(t.n) ? imin(a.sinks, t.n) : 0;  // keys whose gradients have partials
    if (kSink && (n_sink == 0 || t.t0 / a.chunk < a.sink().first_chunk())) return;
    const int c0 = kSink ? (int)(blockIdx.x / slots) * kT : t.t0;
    if (kSink && c0 >= n_sink) return;  // (more sinks than the sequence has)
    const int n_keys = kSink ? n_sink : t.n;
    // query tokens: [q0, q1)
    int q0, q1;
    if (kSink) {
        q0 = imax(t.t0, a.w + 1);
        q1 = imin(t.t0 + a.chunk, t.n);
    } else {
        q0 = c0;
        q1 = (int)min((long long)t.n, (long long)c0 + kT + a.w);
    }
    load_tile(K, [&](int r) -> const float* {
        return c0 + r < t.n ? view_row(a.k, t.batch, hk, t.start + c0 + r) : nullptr;
    });
    load_tile(V, [&](int r) -> const float* {
        return c0 + r < t.n ? view_row(a.v, t.batch, hk, t.start + c0 + r) : nullptr;
    });
    float dk[4][4], dv[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) dk[i][c] = dv[i][c] = 0.f;
    const float sc = a.scale * kLog2e;
    for (int qt = q0; qt < q1; qt += TQ) {
        auto live = [&](int r) { return r < TQ * G && qt + r / G < q1; };
        auto o_off = [&](int r) {
            return (((size_t)t.batch * a.L + t.start + qt + r / G) * a.Hq + hk * G + r % G) * kD;
        };
        __syncthreads();
        load_tile(Q, [&](int r) -> const float* {
            return live(r) ? view_row(a.q, t.batch, hk * G + r % G, t.start + qt + r / G) : nullptr;
        });
        load_tile(dO, [&](int r) -> const float* { return live(r) ? static_cast<const float*>(a.dout) + o_off(r) : nullptr; });
        if (threadIdx.x < kT) {
            const int r = threadIdx.x;
            const size_t at = ((size_t)t.batch * a.Hq + hk * G + r % G) * a.L + t.start + qt + r / G;
            lse_s[r] = live(r) ? a.lse[at] * kLog2e : 0.f;
            delta_s[r] = live(r) ? a.delta[at] : 0.f;
        }
        __syncthreads();
        float s[4][4], dp[4][4];
        tile_nt(s, K, Q, ty, tx);
        tile_nt(dp, V, dO, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = tx + 16 * j, key = c0 + 4 * ty + i, qi = qt + r / G;
                const bool in = qi - key <= a.w;
                const bool vis = live(r) && key < n_keys && key <= qi && in != kSink;
                const float p = vis ? exp2f(fmaf(s[i][j], sc, -lse_s[r])) : 0.f;
                P[(4 * ty + i) * kLd + r] = p;
                S[(4 * ty + i) * kLd + r] = vis ? p * (dp[i][j] - delta_s[r]) : 0.f;
            }
        __syncwarp();
        tile_nn(dv, P, dO, ty, tx);
        tile_nn(dk, S, Q, ty, tx);
    }
    const int seq_start = a.cu ? t.start : t.b * a.L;
    const long long part_row =
        kSink ? a.sink().chunk_row(t.b, seq_start, t.t0 / a.chunk) : a.sink().own(t.b, seq_start);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = c0 + 4 * ty + i;
#pragma unroll
        for (int c = 0; c < 4; ++c) dk[i][c] *= a.scale;
        if (key < n_sink) {
            float* p = a.part + ((size_t)hk * a.sink().rows() + part_row + key) * 2 * kD + 4 * tx;
            store4(p, dk[i]);
            store4(p + kD, dv[i]);
            continue;
        }
        if (kSink || key >= t.rows) continue;
        store4(view_row(a.dk, t.batch, hk, t.start + key) + 4 * tx, dk[i]);
        store4(view_row(a.dv, t.batch, hk, t.start + key) + 4 * tx, dv[i]);
    }
}

// Adds the partial gradients of the sink keys: the window's, then the
// chunks' in order.  One 128-thread block per (key, kv head, sequence).
template <typename T>
__global__ void __launch_bounds__(128) sink_reduce_kernel(const __grid_constant__ WindowArgs a) {
    const int key = blockIdx.x % a.sinks, hk = blockIdx.y, b = blockIdx.x / a.sinks, e = threadIdx.x;
    const int start = a.cu ? iclamp(a.cu[b], 0, a.L) : 0;
    const int n = a.cu ? iclamp(a.cu[b + 1], 0, a.L) - start : (a.lens ? iclamp(a.lens[b], 0, a.L) : a.L);
    if (key >= n || !a.sink().any(n)) return;
    const int seq_start = a.cu ? start : b * a.L;
    const float* p = a.part + ((size_t)hk * a.sink().rows() + key) * 2 * kD + e;
    auto at = [&](long long row) -> const float& { return p[(size_t)row * 2 * kD]; };
    float s = at(a.sink().own(b, seq_start));
    const int first = a.sink().first_chunk(), end = (n - 1) / a.chunk + 1;
    s += at(a.sink().chunk_row(b, seq_start, first));
    // the others, 16 loads at a time in flight
    const int more = end - first - 1;
    const float* next = more > 0 ? &at(a.sink().chunk_row(b, seq_start, first + 1)) : nullptr;
    const size_t step = (size_t)a.sinks * 2 * kD;
    for (int c = 0; c < more; c += 16) {
        float x[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) x[u] = c + u < more ? next[(c + u) * step] : 0.f;
#pragma unroll
        for (int u = 0; u < 16; ++u) s += x[u];
    }
    const lf_heads& v = e < kD ? a.dk : a.dv;
    static_cast<T*>(v.data)[(a.cu ? 0 : b) * v.batch_stride + hk * v.head_stride + (start + key) * v.token_stride +
                            (e & (kD - 1))] = from_f<T>(s);
}

template <typename K>
lf_status set_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess
               ? LF_OK : LF_ERR_CUDA;
}

template <typename K, typename... A>
lf_status launch(K kernel, dim3 grid, int tiles, cudaStream_t stream, const A&... a) {
    const size_t bytes = (size_t)tiles * kTile * sizeof(float);
    lf_status st = set_smem(kernel, bytes);
    if (st != LF_OK) return st;
    kernel<<<grid, kThreads, bytes, stream>>>(a...);
    return cudaGetLastError() == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

}  // namespace

lf_status launch_window_forward_simt(const WindowArgs& a, cudaStream_t stream) {
    const int TQ = kT / a.heads_group();
    return launch(forward_kernel, dim3(token_slots(a.packed(), a.n_seqs, a.L, TQ), a.Hkv), 4, stream, a);
}

lf_status launch_window_backward_simt(const WindowArgs& a, cudaStream_t stream) {
    const int TQ = kT / a.heads_group(), tiles = token_slots(a.packed(), a.n_seqs, a.L, kT);
    const int chunks = a.sinks > 0 ? token_slots(a.packed(), a.n_seqs, a.L, a.chunk) : 0;
    const long long sink_tiles = (long long)chunks * ((a.sinks + kT - 1) / kT);
    if (sink_tiles > INT32_MAX) return LF_ERR_TOO_LARGE;
    lf_status st = launch(dq_kernel, dim3(token_slots(a.packed(), a.n_seqs, a.L, TQ), a.Hkv), 5, stream, a);
    if (st == LF_OK) st = launch(dkv_kernel<false>, dim3(tiles, a.Hkv), 6, stream, a, tiles);
    if (st == LF_OK && a.sinks > 0) {
        st = launch(dkv_kernel<true>, dim3((unsigned)sink_tiles, a.Hkv), 6, stream, a, chunks);
        if (st == LF_OK) st = launch_sink_reduce(a, stream);
    }
    return st;
}

lf_status launch_sink_reduce(const WindowArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)a.n_seqs * a.sinks, a.Hkv);
    if (a.dtype == LF_F16) sink_reduce_kernel<__half><<<grid, 128, 0, stream>>>(a);
    else if (a.dtype == LF_BF16) sink_reduce_kernel<__nv_bfloat16><<<grid, 128, 0, stream>>>(a);
    else sink_reduce_kernel<float><<<grid, 128, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

}  // namespace lf
