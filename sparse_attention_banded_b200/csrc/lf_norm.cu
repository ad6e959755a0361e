// Layer norm over the last dimension, forward and backward, any width up to
// 16384, any row stride, fp32 / fp16 / bf16 with fp32 statistics and
// parameters.
//
//   forward   mean, rstd = 1 / sqrt(var + eps) (population variance),
//             y = (x - mean) rstd gamma + beta
//   backward  xh = (x - mean) rstd, g = dy gamma,
//             dx = rstd (g - mean(g) - xh mean(g xh)),
//             dgamma = sum over rows of dy xh, dbeta = sum of dy
//
// Bound by HBM: one read of each input and one write of each output.  A row
// stays in the registers of a group of 32 to 512 threads, 16 elements each
// (32 above 8192 columns), so the variance is centred on the mean without
// reading the row again; the group's next row is on its way while it works
// on this one.  The backward kernel keeps each thread's share of dgamma and
// dbeta in registers over all rows of its block; a second kernel adds the
// blocks' sums.  All sums have a fixed order (no atomics).
// Measured, forward and backward: 16384 x 1024 bf16 44 us, 3.8 of the 6.6
// TB/s of a copy (168 MB; the second kernel's sums, 5 us, and two rows in
// flight per group in the backward, which registers bound, keep it there);
// 5001 x 1537 fp32, an odd width by single elements, 37 us, 4.1 TB/s.
// Where a thread's part of a row does not fit its registers it spills (bytes
// a thread, TB/s of the pass): forward of 4097 to 8192 columns, 64 registers
// for two blocks of 512 threads per SM, 260 and 612, 1.9 at 8192 x 5120 bf16
// against 3.9 at 8192 x 4096; above 8192 columns backward, 470 to 1040, 1.5
// at 2048 x 16384 bf16; backward of 16-bit rows by single elements, 344 to
// 480 at any width, 0.8 at 8192 x 2050 bf16 against 3.2 with 16-byte loads.
#include "lf_convert.cuh"
#include "lf_tc_tiles.cuh"
#include "lf_window.h"

namespace lf {
namespace {

using sm100::named_bar_sync;

// Element offset of a thread's k-th access of VEC elements.
template <int TPR, int VEC>
__device__ __forceinline__ int col_of(int t, int k) { return (k * TPR + t) * VEC; }

template <typename T, int VEC>
struct Vec;
template <typename T>
struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void zero() { v = from_f<T>(0.f); }
    __device__ __forceinline__ float get(int) const { return to_f(v); }
};
template <>
struct Vec<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float get(int e) const { return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w; }
};
template <typename T>
struct Vec<T, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float get(int e) const {
        const uint32_t u = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
        const float2 f = Pair<T>::unpack(u);
        return (e & 1) ? f.y : f.x;
    }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(Pair<T>::pack(x[0], x[1]), Pair<T>::pack(x[2], x[3]),
                                                  Pair<T>::pack(x[4], x[5]), Pair<T>::pack(x[6], x[7]));
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
        *p = from_f<T>(x[0]);
    }
}

constexpr int kMaxThreads = 512;

template <int TPR>
__host__ __device__ constexpr int block_threads() { return TPR > 256 ? TPR : 256; }

// Sums over the TPR threads of a row, in every thread: s.x and s.y.  Groups
// of several warps meet at a named barrier once per call; `red` holds two
// calls' worth of their warps' sums, used in turn.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 s, float2 (*red)[kMaxThreads / 32], int& turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    }
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5, base = warp / W * W;
        float2* r = red[turn];
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) r[warp] = s;
        named_bar_sync(1 + warp / W, TPR);
        s = r[base];
#pragma unroll
        for (int i = 1; i < W; ++i) {
            s.x += r[base + i].x;
            s.y += r[base + i].y;
        }
    }
    return s;
}

// A thread's part of a row of N elements; zeros past the row.
template <typename T, int TPR, int EPT, int VEC>
struct Part {
    Vec<T, VEC> v[EPT / VEC];
    __device__ __forceinline__ void load(const T* row, int t, int N) {
#pragma unroll
        for (int k = 0; k < EPT / VEC; ++k) {
            const int c = col_of<TPR, VEC>(t, k);
            if (c < N) v[k].load(row + c);
            else v[k].zero();
        }
    }
    __device__ __forceinline__ float2 pair(int p) const {
        if constexpr (VEC == 8) {
            const uint4& u = v[p / 4].v;
            const uint32_t w = p % 4 == 0 ? u.x : p % 4 == 1 ? u.y : p % 4 == 2 ? u.z : u.w;
            return Pair<T>::unpack(w);
        } else {
            return make_float2(v[2 * p / VEC].get(2 * p % VEC), v[(2 * p + 1) / VEC].get((2 * p + 1) % VEC));
        }
    }
};
// The parameter of each of the thread's elements (`none` without).
template <int TPR, int EPT, int VEC>
__device__ __forceinline__ void load_param(float2 (&p)[EPT / 2], const float* src, int t, int N, float none) {
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
        const int c = col_of<TPR, VEC>(t, e / VEC) + e % VEC;
        const float v = src && c < N ? __ldg(src + c) : none;
        if (e % 2) p[e / 2].y = v;
        else p[e / 2].x = v;
    }
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
template <typename T, int TPR, int EPT, int VEC>
__device__ __forceinline__ void store_part(T* row, const float2 (&x)[EPT / 2], int t, int N) {
#pragma unroll
    for (int k = 0; k < EPT / VEC; ++k) {
        const int c = col_of<TPR, VEC>(t, k);
        if (c < N) {
            float y[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = (k * VEC + e) % 2 ? x[(k * VEC + e) / 2].y : x[(k * VEC + e) / 2].x;
            store_vec<T, VEC>(row + c, y);
        }
    }
}

template <typename T, int TPR, int EPT, int VEC>
__global__ void __launch_bounds__(block_threads<TPR>(), TPR * EPT > 8192 ? 1 : 2)
forward_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kRows = block_threads<TPR>() / TPR;
    __shared__ float2 red[2][kMaxThreads / 32];
    sm100::pdl_launch_dependents();
    sm100::pdl_wait();
    const int t = threadIdx.x % TPR;
    const unsigned step = gridDim.x * kRows, rows = a.rows;
    const T* x = static_cast<const T*>(a.x);
    int turn = 0;
    unsigned row = blockIdx.x * kRows + threadIdx.x / TPR;  // (row + kDepth steps stay below 2^32)
    if (row >= rows) return;
    constexpr int kDepth = sizeof(T) * EPT <= 32 ? 4 : 2;  // rows in flight
    Part<T, TPR, EPT, VEC> buf[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if (row + d * step < rows) buf[d].load(x + (row + d * step) * a.x_stride, t, a.N);
    float2 gamma[EPT / 2], beta[EPT / 2];
    load_param<TPR, EPT, VEC>(gamma, a.gamma, t, a.N, 1.f);
    load_param<TPR, EPT, VEC>(beta, a.beta, t, a.N, 0.f);
    const float inv_n = 1.f / (float)a.N;
    // Pairs in packed fp32 arithmetic: with 16-bit elements the instructions,
    // not the loads, would bound one row after another.
    while (row < rows) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d, row += step) {
            if (row >= rows) break;
            auto& cur = buf[d];
            float2 c[EPT / 2], s = both(0.f);
#pragma unroll
            for (int p = 0; p < EPT / 2; ++p) {
                c[p] = cur.pair(p);
                s = fadd2(s, c[p]);
            }
            const float mean = row_sum<TPR>(make_float2(s.x + s.y, 0.f), red, turn).x * inv_n;
            float2 q = both(0.f);
#pragma unroll
            for (int p = 0; p < EPT / 2; ++p) {
                c[p] = fadd2(c[p], both(-mean));
                // past the row: not counted
                const int c0 = col_of<TPR, VEC>(t, 2 * p / VEC), c1 = col_of<TPR, VEC>(t, (2 * p + 1) / VEC);
                const float2 z = make_float2(c0 < a.N ? c[p].x : 0.f, c1 < a.N ? c[p].y : 0.f);
                q = ffma2(z, z, q);
            }
            const float var = row_sum<TPR>(make_float2(q.x + q.y, 0.f), red, turn).x * inv_n;
            const float rstd = 1.f / sqrtf(var + a.eps);
            if (t == 0) {
                if (a.mean) a.mean[row] = mean;
                if (a.rstd) a.rstd[row] = rstd;
            }
#pragma unroll
            for (int p = 0; p < EPT / 2; ++p) c[p] = ffma2(fmul2(c[p], both(rstd)), gamma[p], beta[p]);
            store_part<T, TPR, EPT, VEC>(static_cast<T*>(a.y) + (long long)row * a.N, c, t, a.N);
            const unsigned ahead = row + kDepth * step;
            if (ahead < rows) cur.load(x + ahead * a.x_stride, t, a.N);
        }
    }
}

template <typename T, int TPR, int EPT, int VEC>
__global__ void __launch_bounds__(block_threads<TPR>(), TPR > 256 ? 1 : 2)
backward_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kRows = block_threads<TPR>() / TPR;
    extern __shared__ float sums[];  // [kRows - 1][EPT][TPR] for the block's reduction
    __shared__ float2 red[2][kMaxThreads / 32];
    sm100::pdl_launch_dependents();
    sm100::pdl_wait();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const unsigned step = gridDim.x * kRows, rows = a.rows;
    const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(a.dy);
    float2 dg[EPT / 2], db[EPT / 2], gamma[EPT / 2];
#pragma unroll
    for (int p = 0; p < EPT / 2; ++p) dg[p] = db[p] = both(0.f);
    load_param<TPR, EPT, VEC>(gamma, a.gamma, t, a.N, 1.f);
    const float inv_n = 1.f / (float)a.N;
    int turn = 0;
    unsigned row = blockIdx.x * kRows + grp;  // (row + kDepth steps stay below 2^32)
    constexpr int kDepth = sizeof(T) * EPT <= 32 ? 2 : 1;  // rows in flight
    Part<T, TPR, EPT, VEC> xb[kDepth], yb[kDepth];
    float mean_b[kDepth], rstd_b[kDepth];
    auto fetch = [&](int d, unsigned r) {
        xb[d].load(x + r * a.x_stride, t, a.N);
        yb[d].load(dy + r * a.dy_stride, t, a.N);
        mean_b[d] = a.mean[r];
        rstd_b[d] = a.rstd[r];
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if (row + d * step < rows) fetch(d, row + d * step);
    while (row < rows) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d, row += step) {
            if (row >= rows) break;
            const float rstd = rstd_b[d];
            const float2 nmean = both(-mean_b[d]), rs = both(rstd);
            float2 xh[EPT / 2], g[EPT / 2], s1 = both(0.f), s2 = both(0.f);  // sums of g and of g xh
#pragma unroll
            for (int p = 0; p < EPT / 2; ++p) {  // (past the row dy is 0)
                const float2 v = yb[d].pair(p);
                xh[p] = fmul2(fadd2(xb[d].pair(p), nmean), rs);
                g[p] = fmul2(v, gamma[p]);
                s1 = fadd2(s1, g[p]);
                s2 = ffma2(g[p], xh[p], s2);
                dg[p] = ffma2(v, xh[p], dg[p]);
                db[p] = fadd2(db[p], v);
            }
            const unsigned ahead = row + kDepth * step;
            if (ahead < rows) fetch(d, ahead);
            const float2 s = row_sum<TPR>(make_float2(s1.x + s1.y, s2.x + s2.y), red, turn);
            const float2 nm1 = both(-s.x * inv_n * rstd), nm2 = both(-s.y * inv_n * rstd);
#pragma unroll
            for (int p = 0; p < EPT / 2; ++p) g[p] = ffma2(xh[p], nm2, ffma2(g[p], rs, nm1));
            store_part<T, TPR, EPT, VEC>(static_cast<T*>(a.y) + (long long)row * a.N, g, t, a.N);
        }
    }
    if (!a.part) return;
    // the block's row groups, added in order by the first
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        float acc[EPT];
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            const float2 v = pass ? db[e / 2] : dg[e / 2];
            acc[e] = e % 2 ? v.y : v.x;
        }
        if constexpr (kRows > 1) {
            __syncthreads();
            if (grp > 0)
#pragma unroll
                for (int e = 0; e < EPT; ++e) sums[((grp - 1) * EPT + e) * TPR + t] = acc[e];
            __syncthreads();
            if (grp == 0)
#pragma unroll
                for (int e = 0; e < EPT; ++e)
                    for (int u = 0; u < kRows - 1; ++u) acc[e] += sums[(u * EPT + e) * TPR + t];
        }
        if (grp == 0) {
            float* p = a.part + ((size_t)blockIdx.x * 2 + pass) * a.N;
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                const int c = col_of<TPR, VEC>(t, e / VEC) + e % VEC;
                if (c < a.N) p[c] = acc[e];
            }
        }
    }
}

// dgamma / dbeta: column sums of the blocks' partial rows.  32 columns x 32
// groups of partial rows per block, each group's loads in flight together;
// the groups' sums are joined by a fixed tree.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ part, int blocks, int N,
                                                          float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ float s[32][33];
    sm100::pdl_wait();
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int which = blockIdx.y;
    float* out = which ? dbeta : dgamma;
    if (!out) return;
    float acc = 0.f;
    if (c < N) {
#pragma unroll 10
        for (int b = grp; b < blocks; b += 32) acc += part[((size_t)b * 2 + which) * N + c];
    }
    s[grp][lane] = acc;
    __syncthreads();
    // warp g joins the groups' sums of column g
    acc = s[lane][grp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    const int col = blockIdx.x * 32 + grp;
    if (lane == 0 && col < N) out[col] = acc;
}

// Threads per row: the narrowest group whose registers hold the row.
int threads_per_row(int N) {
    int t = 32;
    while (t < 512 && t * 16 < N) t *= 2;
    return t;
}

// Blocks of the backward kernel: two per SM of a B200, fewer for few rows.
constexpr int kMaxBlocks = 2 * 148;
int backward_blocks(int rows, int N) {
    const int tpr = threads_per_row(N), per = tpr > 256 ? 1 : 256 / tpr;
    return imin((rows - 1) / per + 1, kMaxBlocks);  // (rows > 0, up to 2^31 - 1)
}

template <typename T, int TPR, int EPT, int VEC>
lf_status run_forward(const NormArgs& a, cudaStream_t stream) {
    constexpr int kRows = block_threads<TPR>() / TPR;
    const int blocks = imin((a.rows - 1) / kRows + 1, 2 * 148);
    return launch_pdl(forward_kernel<T, TPR, EPT, VEC>, dim3(blocks), dim3(block_threads<TPR>()), 0, stream, a);
}

template <typename T, int TPR, int EPT, int VEC>
lf_status run_backward(const NormArgs& a, cudaStream_t stream) {
    constexpr int kRows = block_threads<TPR>() / TPR;
    constexpr size_t bytes = (size_t)(kRows - 1) * TPR * EPT * sizeof(float);
    static_assert(bytes <= 48 * 1024 - 512, "the block's reduction");
    return launch_pdl(backward_kernel<T, TPR, EPT, VEC>, dim3(backward_blocks(a.rows, a.N)), dim3(block_threads<TPR>()),
                      bytes, stream, a);
}

// 16-byte accesses where every row starts on a 16-byte boundary.
bool wide(const NormArgs& a, bool backward) {
    const int per = a.dtype == LF_F32 ? 4 : 8;
    return a.N % per == 0 && a.x_stride % per == 0 && (!backward || a.dy_stride % per == 0);
}

template <bool kBack, typename T, int TPR, int EPT>
lf_status run_vec(const NormArgs& a, cudaStream_t stream) {
    constexpr int kWide = sizeof(T) == 4 ? 4 : 8;
    if constexpr (kBack)
        return wide(a, true) ? run_backward<T, TPR, EPT, kWide>(a, stream) : run_backward<T, TPR, EPT, 1>(a, stream);
    else
        return wide(a, false) ? run_forward<T, TPR, EPT, kWide>(a, stream) : run_forward<T, TPR, EPT, 1>(a, stream);
}
template <bool kBack, typename T>
lf_status run_tpr(const NormArgs& a, cudaStream_t stream) {
    switch (threads_per_row(a.N)) {
        case 32: return run_vec<kBack, T, 32, 16>(a, stream);
        case 64: return run_vec<kBack, T, 64, 16>(a, stream);
        case 128: return run_vec<kBack, T, 128, 16>(a, stream);
        case 256: return run_vec<kBack, T, 256, 16>(a, stream);
        default: return a.N <= 512 * 16 ? run_vec<kBack, T, 512, 16>(a, stream) : run_vec<kBack, T, 512, 32>(a, stream);
    }
}
template <bool kBack>
lf_status run_dtype(const NormArgs& a, cudaStream_t stream) {
    if (a.dtype == LF_F16) return run_tpr<kBack, __half>(a, stream);
    if (a.dtype == LF_BF16) return run_tpr<kBack, __nv_bfloat16>(a, stream);
    return run_tpr<kBack, float>(a, stream);
}

}  // namespace

size_t norm_backward_bytes(int rows, int N) {
    return (size_t)backward_blocks(rows, N) * 2 * N * sizeof(float);
}

lf_status launch_norm_forward(const NormArgs& a, cudaStream_t stream) { return run_dtype<false>(a, stream); }

lf_status launch_norm_backward(const NormArgs& a, cudaStream_t stream) {
    lf_status st = run_dtype<true>(a, stream);
    if (st != LF_OK || !a.part) return st;
    return launch_pdl(column_sum_kernel, dim3((a.N + 31) / 32, 2), dim3(1024), 0, stream, a.part,
                      backward_blocks(a.rows, a.N), a.N, a.dgamma, a.dbeta);
}

}  // namespace lf
