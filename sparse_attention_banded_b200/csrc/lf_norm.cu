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
// stays in the registers of 32, 128 or 512 threads (32 elements each), so
// the variance is centred on the mean without reading the row again.  The
// backward kernel keeps each thread's share of dgamma and dbeta in registers
// over all rows of its block; a second kernel adds the blocks' sums.  All
// sums have a fixed order (no atomics).
#include "lf_convert.cuh"
#include "lf_window.h"

namespace lf {
namespace {

constexpr int kEpt = 32;  // elements per thread

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

// Sums of a and b over the TPR threads of a row, in every thread.  `red`:
// shared memory for 2 floats per warp of the block.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 s, float2* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    }
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5, base = warp / W * W;
        __syncthreads();  // the previous sum has been read
        if ((threadIdx.x & 31) == 0) red[warp] = s;
        __syncthreads();
        s = red[base];
#pragma unroll
        for (int i = 1; i < W; ++i) {
            s.x += red[base + i].x;
            s.y += red[base + i].y;
        }
    }
    return s;
}

template <int TPR>
constexpr int block_threads() { return TPR > 256 ? TPR : 256; }

template <typename T, int TPR, int VEC>
__global__ void __launch_bounds__(block_threads<TPR>()) forward_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kAcc = kEpt / VEC, kRows = block_threads<TPR>() / TPR;
    __shared__ float2 red[block_threads<TPR>() / 32];
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = row < a.rows;
    const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.x_stride;
    Vec<T, VEC> v[kAcc];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kAcc; ++k) {
        const int c = col_of<TPR, VEC>(t, k);
        if (live && c < a.N) v[k].load(x + c);
        else v[k].zero();
    }
#pragma unroll
    for (int k = 0; k < kAcc; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += v[k].get(e);
    const float mean = row_sum<TPR>(make_float2(s, 0.f), red).x / (float)a.N;
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < kAcc; ++k)
        if (col_of<TPR, VEC>(t, k) < a.N) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = v[k].get(e) - mean;
                q = fmaf(d, d, q);
            }
        }
    const float var = row_sum<TPR>(make_float2(q, 0.f), red).x / (float)a.N;
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (!live) return;
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.N;
#pragma unroll
    for (int k = 0; k < kAcc; ++k) {
        const int c = col_of<TPR, VEC>(t, k);
        if (c >= a.N) continue;
        Vec<float, VEC == 8 ? 4 : VEC> g[VEC == 8 ? 2 : 1], b[VEC == 8 ? 2 : 1];
        constexpr int kHalf = VEC == 8 ? 4 : VEC;
#pragma unroll
        for (int u = 0; u < VEC / kHalf; ++u) {
            if (a.gamma) g[u].load(a.gamma + c + u * kHalf);
            if (a.beta) b[u].load(a.beta + c + u * kHalf);
        }
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            o[e] = fmaf((v[k].get(e) - mean) * rstd, a.gamma ? g[e / kHalf].get(e % kHalf) : 1.f,
                        a.beta ? b[e / kHalf].get(e % kHalf) : 0.f);
        store_vec<T, VEC>(y + c, o);
    }
}

template <typename T, int TPR, int VEC>
__global__ void __launch_bounds__(block_threads<TPR>()) backward_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kAcc = kEpt / VEC, kRows = block_threads<TPR>() / TPR;
    extern __shared__ float sums[];  // [kRows - 1][TPR][kEpt] for the block's reduction
    __shared__ float2 red[block_threads<TPR>() / 32];
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    float dg[kEpt], db[kEpt];
#pragma unroll
    for (int e = 0; e < kEpt; ++e) dg[e] = db[e] = 0.f;
    for (long long r0 = (long long)blockIdx.x * kRows; r0 < a.rows; r0 += (long long)gridDim.x * kRows) {
        const long long row = r0 + grp;
        const bool live = row < a.rows;
        const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.x_stride;
        const T* dy = static_cast<const T*>(a.dy) + (live ? row : 0) * a.dy_stride;
        const float mean = live ? a.mean[row] : 0.f, rstd = live ? a.rstd[row] : 0.f;
        Vec<T, VEC> xv[kAcc], dv[kAcc];
#pragma unroll
        for (int k = 0; k < kAcc; ++k) {
            const int c = col_of<TPR, VEC>(t, k);
            if (live && c < a.N) {
                xv[k].load(x + c);
                dv[k].load(dy + c);
            } else {
                xv[k].zero();
                dv[k].zero();
            }
        }
        float2 s = make_float2(0.f, 0.f);  // sums of g and of g xh
#pragma unroll
        for (int k = 0; k < kAcc; ++k) {
            const int c = col_of<TPR, VEC>(t, k);
            if (!live || c >= a.N) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = dv[k].get(e), xh = (xv[k].get(e) - mean) * rstd;
                const float g = a.gamma ? d * __ldg(a.gamma + c + e) : d;
                s.x += g;
                s.y = fmaf(g, xh, s.y);
                dg[k * VEC + e] = fmaf(d, xh, dg[k * VEC + e]);
                db[k * VEC + e] += d;
            }
        }
        s = row_sum<TPR>(s, red);
        if (!live) continue;
        const float m1 = s.x / (float)a.N, m2 = s.y / (float)a.N;
        T* dx = static_cast<T*>(a.y) + row * a.N;
#pragma unroll
        for (int k = 0; k < kAcc; ++k) {
            const int c = col_of<TPR, VEC>(t, k);
            if (c >= a.N) continue;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = dv[k].get(e), xh = (xv[k].get(e) - mean) * rstd;
                const float g = a.gamma ? d * __ldg(a.gamma + c + e) : d;
                o[e] = rstd * (g - m1 - xh * m2);
            }
            store_vec<T, VEC>(dx + c, o);
        }
    }
    if (!a.part) return;
    // the block's row groups, added in order by the first
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        float (&acc)[kEpt] = pass ? db : dg;
        if constexpr (kRows > 1) {
            __syncthreads();
            if (grp > 0)
#pragma unroll
                for (int e = 0; e < kEpt; ++e) sums[((grp - 1) * kEpt + e) * TPR + t] = acc[e];
            __syncthreads();
            if (grp == 0)
#pragma unroll
                for (int e = 0; e < kEpt; ++e)
                    for (int u = 0; u < kRows - 1; ++u) acc[e] += sums[(u * kEpt + e) * TPR + t];
        }
        if (grp == 0) {
            float* p = a.part + ((size_t)blockIdx.x * 2 + pass) * a.N;
#pragma unroll
            for (int k = 0; k < kAcc; ++k)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int c = col_of<TPR, VEC>(t, k) + e;
                    if (c < a.N) p[c] = acc[k * VEC + e];
                }
        }
    }
}

// dgamma / dbeta: column sums of the blocks' partial rows.  32 columns x 8
// row groups per block, groups added in order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ part, int blocks, int N,
                                                         float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int which = blockIdx.y;
    float* out = which ? dbeta : dgamma;
    if (!out) return;
    float acc = 0.f;
    if (c < N)
        for (int b = grp; b < blocks; b += 8) acc += part[((size_t)b * 2 + which) * N + c];
    s[grp][lane] = acc;
    __syncthreads();
    if (grp == 0 && c < N) {
        for (int g = 1; g < 8; ++g) acc += s[g][lane];
        out[c] = acc;
    }
}

// Threads per row: the narrowest group whose registers hold the row.
int threads_per_row(int N) { return N <= 32 * kEpt ? 32 : N <= 128 * kEpt ? 128 : 512; }

// Blocks of the backward kernel: two per SM of a B200, fewer for few rows.
constexpr int kMaxBlocks = 2 * 148;
int backward_blocks(int rows, int N) {
    const int tpr = threads_per_row(N), per = tpr > 256 ? 1 : 256 / tpr;
    return imin((rows + per - 1) / per, kMaxBlocks);
}

template <typename T, int TPR, int VEC>
lf_status run_forward(const NormArgs& a, cudaStream_t stream) {
    constexpr int kRows = block_threads<TPR>() / TPR;
    forward_kernel<T, TPR, VEC><<<(a.rows + kRows - 1) / kRows, block_threads<TPR>(), 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

template <typename T, int TPR, int VEC>
lf_status run_backward(const NormArgs& a, cudaStream_t stream) {
    constexpr int kRows = block_threads<TPR>() / TPR;
    constexpr size_t bytes = (size_t)(kRows - 1) * TPR * kEpt * sizeof(float);
    if (bytes > 48 * 1024 && cudaFuncSetAttribute(backward_kernel<T, TPR, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  (int)bytes) != cudaSuccess)
        return LF_ERR_CUDA;
    backward_kernel<T, TPR, VEC><<<backward_blocks(a.rows, a.N), block_threads<TPR>(), bytes, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

// 16-byte accesses where every row starts on a 16-byte boundary.
bool wide(const NormArgs& a, bool backward) {
    const int per = a.dtype == LF_F32 ? 4 : 8;
    return a.N % per == 0 && a.x_stride % per == 0 && (!backward || a.dy_stride % per == 0);
}

template <bool kBack, typename T, int TPR>
lf_status run_vec(const NormArgs& a, cudaStream_t stream) {
    constexpr int kWide = sizeof(T) == 4 ? 4 : 8;
    if constexpr (kBack)
        return wide(a, true) ? run_backward<T, TPR, kWide>(a, stream) : run_backward<T, TPR, 1>(a, stream);
    else
        return wide(a, false) ? run_forward<T, TPR, kWide>(a, stream) : run_forward<T, TPR, 1>(a, stream);
}
template <bool kBack, typename T>
lf_status run_tpr(const NormArgs& a, cudaStream_t stream) {
    switch (threads_per_row(a.N)) {
        case 32: return run_vec<kBack, T, 32>(a, stream);
        case 128: return run_vec<kBack, T, 128>(a, stream);
        default: return run_vec<kBack, T, 512>(a, stream);
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
    column_sum_kernel<<<dim3((a.N + 31) / 32, 2), 256, 0, stream>>>(a.part, backward_blocks(a.rows, a.N),
                                                                    a.N, a.dgamma, a.dbeta);
    return cudaGetLastError() == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

}  // namespace lf
