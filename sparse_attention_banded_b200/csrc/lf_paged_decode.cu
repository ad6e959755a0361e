// Paged attention of few new tokens (at most 16 query rows per key/value
// head: tokens x grouped heads), and the merge of split contexts.
//
// Bound by HBM: each visible key and value is read once, 256 bytes for at
// most 4 * 64 * 16 flops.  The keys of a sequence are listed as tiles of 8
// (the sinks', then the window's; a tile lies in one page) and cut into
// chunks, one CTA per (chunk, key/value head, sequence); its four warps take
// 32 keys at a time and keep 8 KB in flight each, with no shared memory in
// the way: the MMA's contraction index may be permuted as long as both
// operands agree, so the 16-byte pieces of a K row a lane loads are its
// mma.m16n8k16 fragments as they stand, and of V rows two keys' words are
// interleaved by byte permutes.  (These are memory-bound 16-row products;
// tcgen05 tiles have 128 rows.)
//
// 48 tokens over contexts to 8192, 16 / 4 heads, bf16: 44 us, 4.4 TB/s of the
// 6.6 of a copy, and 54 us with the keys through shared memory by TMA (a CTA
// then holds fewer bytes in flight than its registers do).
//
// Each warp runs an online softmax over its keys; the warps' results are
// joined in shared memory, the chunks' by the merge kernel: with the log2-
// sum-exp e_s and normalised row o_s of chunk s,
//     out = sum_s 2^(e_s - max e) o_s / sum_s 2^(e_s - max e).
#include "lf_paged_split.h"
#include "lf_tc_tiles.cuh"

namespace lf {
namespace {

using namespace sm100;

constexpr int kWarps = 4;
constexpr int kRows = kDecodeRows;  // 16
constexpr int kD = 64;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// 16 bytes, read once: not kept in L1.
__device__ __forceinline__ uint4 ldg16(const void* p) {
    uint4 v;
    asm("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 3)
decode_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedPlan pl) {
    extern __shared__ int2 tiles[];  // [chunk] (position, page)
    __shared__ float o_s[kWarps][kRows][kD + 4];
    __shared__ float ml_s[kWarps][kRows][2];
    const int b = blockIdx.x / pl.decode_splits, piece = blockIdx.x % pl.decode_splits, hk = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0 && hk == 0) check_lengths(a.cu, nullptr, a.n_seqs, a.T, a.status, threadIdx.x, blockDim.x);
    const int start = iclamp(a.cu[b], 0, a.T), n = iclamp(a.cu[b + 1], 0, a.T) - start, G = a.Hq / a.Hkv;
    int kv, first;
    if (n <= 0 || !paged_seq(a, b, n, kv, first, threadIdx.x == 0 && hk == 0 && piece == 0)) return;
    if (n * G > kRows) return;  // the tensor-core kernel's
    const KeyBlocks kb = decode_tiles(first, n, kv, a.w, a.sinks);
    const int t0 = piece * pl.chunk, t1 = imin(t0 + pl.chunk, kb.n);
    T* out = static_cast<T*>(a.out);
    if (t0 >= t1) {
        if (piece == 0)  // no key at all
            for (int e = threadIdx.x; e < n * G * 8; e += kWarps * 32) {
                const int r = e >> 3;
                reinterpret_cast<uint4*>(out + ((size_t)(start + r / G) * a.Hq + hk * G + r % G) * kD)[e & 7] =
                    make_uint4(0u, 0u, 0u, 0u);
            }
        return;
    }
    const int i0 = imax(first, 0), i1 = first + n - 1;
    for (int t = threadIdx.x; t < t1 - t0; t += kWarps * 32) {
        const int pos = key_block(kb, t0 + t) * 8;
        const int page = page_of(a.table + (size_t)b * a.max_pages, a.max_pages, a.num_pages, a.page_shift, pos);
        if (page < 0 && range_visible(i0, i1, pos, imin(pos + 8, kv) - 1, a.w, a.sinks))
            record_status(a.status, b, LF_ERR_BAD_PAGE);
        tiles[t] = make_int2(pos, page);
    }
    const int g = lane >> 2, t4 = lane & 3;  // fragment row / column group
    // Q: rows g and g + 8, the 16 elements of the head dim this lane's K
    // pieces hold: 8 t4 .. and 32 + 8 t4 ..
    uint32_t q[4][4];
    int pos_row[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = g + 8 * u;
        const bool live = r < n * G;
        pos_row[u] = live ? first + r / G : -1;
        const T* p = view_row<T>(a.q, 0, hk * G + (live ? r % G : 0), start + (live ? r / G : 0)) + 8 * t4;
        const uint4 lo = live ? ldg16(p) : make_uint4(0u, 0u, 0u, 0u), hi = live ? ldg16(p + 32) : make_uint4(0u, 0u, 0u, 0u);
        q[0][u] = lo.x; q[0][u + 2] = lo.y;
        q[1][u] = lo.z; q[1][u + 2] = lo.w;
        q[2][u] = hi.x; q[2][u + 2] = hi.y;
        q[3][u] = hi.z; q[3][u + 2] = hi.w;
    }
    __syncthreads();

    const float sc = a.scale * kLog2e;
    float o[8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    const int in_page = (1 << a.page_shift) - 1;
    const T* kbase = static_cast<const T*>(a.k.data) + hk * a.k.head_stride + 8 * t4;
    const T* vbase = static_cast<const T*>(a.v.data) + hk * a.v.head_stride + 8 * g;

    for (int t = t0 + 4 * warp; t < t1; t += 4 * kWarps) {
        uint4 kx[4][2], vx[4][2];  // K: tile, piece.  V: tile, key 2 t4 / 2 t4 + 1
        int2 tl[4];
        bool part = false;         // some key of the four tiles is seen by no row, or missing
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            tl[u] = t + u < t1 ? tiles[t - t0 + u] : make_int2(0, -1);
            const int pos = tl[u].x, slot = pos & in_page;
            part |= tl[u].y < 0 || !block_full(i0, i1, pos, 8, kv, a.w, a.sinks) || first < 0;
            if (tl[u].y >= 0) {
                const T* kp = kbase + tl[u].y * a.k.batch_stride + (slot + g) * a.k.token_stride;
                const T* vp = vbase + tl[u].y * a.v.batch_stride + (slot + 2 * t4) * a.v.token_stride;
                kx[u][0] = ldg16(kp);
                kx[u][1] = ldg16(kp + 32);
                vx[u][0] = ldg16(vp);
                vx[u][1] = ldg16(vp + a.v.token_stride);
            } else {
                kx[u][0] = kx[u][1] = vx[u][0] = vx[u][1] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        float s[4][4];
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
            mma16816<T>(s[u], q[0], kx[u][0].x, kx[u][0].y);
            mma16816<T>(s[u], q[1], kx[u][0].z, kx[u][0].w);
            mma16816<T>(s[u], q[2], kx[u][1].x, kx[u][1].y);
            mma16816<T>(s[u], q[3], kx[u][1].z, kx[u][1].w);
            if (part) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = tl[u].x + 2 * t4 + (e & 1);
                    const bool vis = tl[u].y >= 0 && key < kv && key_visible(pos_row[e >> 1], key, a.w, a.sinks);
                    s[u][e] = vis ? s[u][e] : -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // 0 * NaN: rows of V that no query sees
                    const int key = tl[u].x + 2 * t4 + e;
                    if (key >= kv || !range_visible(i0, i1, key, key, a.w, a.sinks)) vx[u][e] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            mx[0] = max3(mx[0], s[u][0], s[u][1]);
            mx[1] = max3(mx[1], s[u][2], s[u][3]);
        }
        float f[2], nm[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
            mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
            const float mn = fmaxf(m[u], mx[u] * sc);
            nm[u] = mn == -INFINITY ? 0.f : -mn;
            f[u] = ex2(m[u] + nm[u]);
            m[u] = mn;
            l[u] *= f[u];
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            o[c][0] *= f[0];
            o[c][1] *= f[0];
            o[c][2] *= f[1];
            o[c][3] *= f[1];
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            // P of 16 keys: rounded to the storage type, the MMA's operand type
            uint32_t p[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* x = s[2 * v + h];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = ex2(fmaf(x[e], sc, nm[e >> 1]));
                l[0] += x[0] + x[1];
                l[1] += x[2] + x[3];
                p[2 * h] = Pair<T>::pack(x[0], x[1]);
                p[2 * h + 1] = Pair<T>::pack(x[2], x[3]);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                // column g of the c-th product is element 8 g + c of the head dim
                const uint32_t sel = (c & 1) ? 0x7632u : 0x5410u;
                const uint32_t b0 = __byte_perm(word(vx[2 * v][0], c >> 1), word(vx[2 * v][1], c >> 1), sel);
                const uint32_t b1 = __byte_perm(word(vx[2 * v + 1][0], c >> 1), word(vx[2 * v + 1][1], c >> 1), sel);
                mma16816<T>(o[c], p, b0, b1);
            }
        }
    }
    // the warps' rows
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
        const int r = g + 8 * u;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float* d = &o_s[warp][r][8 * (2 * t4 + e)];
            *reinterpret_cast<float4*>(d) = make_float4(o[0][2 * u + e], o[1][2 * u + e], o[2][2 * u + e], o[3][2 * u + e]);
            *reinterpret_cast<float4*>(d + 4) = make_float4(o[4][2 * u + e], o[5][2 * u + e], o[6][2 * u + e], o[7][2 * u + e]);
        }
        if (t4 == 0) {
            ml_s[warp][r][0] = m[u];
            ml_s[warp][r][1] = l[u];
        }
    }
    __syncthreads();
    const bool whole = kb.n <= pl.chunk;  // one chunk holds every key
    for (int e = threadIdx.x; e < n * G * 8; e += kWarps * 32) {
        const int r = e >> 3, c = (e & 7) * 8;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml_s[w][r][0]);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(ml_s[w][r][0] - base);
            sum = fmaf(f, ml_s[w][r][1], sum);
#pragma unroll
            for (int d = 0; d < 8; ++d) x[d] = fmaf(f, o_s[w][r][c + d], x[d]);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int d = 0; d < 8; ++d) x[d] *= inv;
        const int head = hk * G + r % G;
        if (whole) {
            const size_t row = (size_t)(start + r / G) * a.Hq + head;
            reinterpret_cast<uint4*>(out + row * kD)[e & 7] = make_uint4(
                Pair<T>::pack(x[0], x[1]), Pair<T>::pack(x[2], x[3]), Pair<T>::pack(x[4], x[5]), Pair<T>::pack(x[6], x[7]));
        } else {
            const size_t at = ((size_t)piece * pl.decode_tokens + pl.decode_slot(b, start, r / G)) * a.Hq + head;
            float4* d = reinterpret_cast<float4*>(pl.decode_o() + at * kD + c);
            d[0] = make_float4(x[0], x[1], x[2], x[3]);
            d[1] = make_float4(x[4], x[5], x[6], x[7]);
            if (c == 0) pl.decode_lse(a.T, a.Hq)[at] = sum == 0.f ? -INFINITY : top + log2f(sum);
        }
    }
}

// Partials of one row: the weighted sum of some of them, 4 elements a lane.
struct Joined {
    float top, sum;
    float4 x;
};
// `count` partials `step` rows apart, every `stride`-th from `from` on; o:
// this lane's elements of the first.
__device__ __forceinline__ Joined join(const float* o, const float* e, size_t step, int count, int from, int stride) {
    Joined j = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
    for (int s = from; s < count; s += stride) j.top = fmaxf(j.top, e[s * step]);
    const float base = j.top == -INFINITY ? 0.f : j.top;
#pragma unroll 4
    for (int s = from; s < count; s += stride) {
        const float f = ex2(e[s * step] - base);
        const float4 v = *reinterpret_cast<const float4*>(o + s * step * kD);
        j.sum += f;
        j.x = make_float4(fmaf(f, v.x, j.x.x), fmaf(f, v.y, j.x.y), fmaf(f, v.z, j.x.z), fmaf(f, v.w, j.x.w));
    }
    return j;
}
__device__ __forceinline__ Joined join2(const Joined& a, const Joined& b) {
    Joined j;
    j.top = fmaxf(a.top, b.top);
    const float base = j.top == -INFINITY ? 0.f : j.top, fa = ex2(a.top - base), fb = ex2(b.top - base);
    j.sum = a.sum * fa + b.sum * fb;
    j.x = make_float4(a.x.x * fa + b.x.x * fb, a.x.y * fa + b.x.y * fb, a.x.z * fa + b.x.z * fb, a.x.w * fa + b.x.w * fb);
    return j;
}

// Joins the pieces of rows that have several, half a warp per row.  kBlock:
// the 16 half warps of a block share one row (a context may be cut into many
// pieces); else a warp takes kEach heads of one token, two at a time, and
// looks its sequence up once.
template <typename T, bool kBlock, int kEach>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedPlan pl) {
    __shared__ Joined parts[16][16];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1, G = a.Hq / a.Hkv;
    const int each = (a.Hq + kEach - 1) / kEach;  // warps (blocks) per token
    const long long at = kBlock ? blockIdx.x : (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (at >= (long long)a.T * each) return;
    const int tok = (int)(at / each), h0 = (int)(at % each) * kEach;
    const int b = seq_of_token_warp(a.cu, a.n_seqs, tok);
    const int start = iclamp(a.cu[b], 0, a.T), n = iclamp(a.cu[b + 1], 0, a.T) - start;
    if (tok < start || tok >= start + n) return;
    int kv, first;
    if (!paged_seq(a, b, n, kv, first, false)) return;
    // the pieces: how many, how many rows apart, where this token's are
    int pieces;
    const float *po, *pe;
    size_t step, at0;
    if (pl.decode && n * G <= kRows) {
        pieces = (decode_tiles(first, n, kv, a.w, a.sinks).n + pl.chunk - 1) / pl.chunk;
        po = pl.decode_o();
        pe = pl.decode_lse(a.T, a.Hq);
        step = (size_t)pl.decode_tokens * a.Hq;
        at0 = (size_t)pl.decode_slot(b, start, tok - start) * a.Hq + h0;
    } else {
        const int TQ = 128 / G, t0 = (tok - start) / TQ * TQ;
        pieces = (tile_key_blocks(first, t0, imin(t0 + TQ, n), kv, a.w, a.sinks).n + pl.per - 1) / pl.per;
        po = pl.o(a.Hq);
        pe = pl.lse(a.T, a.Hq);
        step = (size_t)a.T * a.Hq;
        at0 = (size_t)tok * a.Hq + h0;
    }
    if (pieces <= 1) return;  // written whole
    const size_t row0 = (size_t)tok * a.Hq + h0;
    auto store = [&](const Joined& j, size_t row) {
        const float inv = j.sum == 0.f ? 0.f : 1.f / j.sum;
        reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * kD)[lane] =
            make_uint2(Pair<T>::pack(j.x.x * inv, j.x.y * inv), Pair<T>::pack(j.x.z * inv, j.x.w * inv));
    };
    if constexpr (kBlock) {
        static_assert(kEach == 1, "one row per block");
        const int part = threadIdx.x >> 4;
        parts[part][lane] = join(po + at0 * kD + 4 * lane, pe + at0, step, pieces, part, 16);
        __syncthreads();
        if (part > 0) return;
        Joined j = parts[0][lane];
        for (int u = 1; u < 16; ++u) j = join2(j, parts[u][lane]);
        store(j, row0);
    } else {
#pragma unroll
        for (int h = half; h < kEach; h += 2)
            if (h0 + h < a.Hq) store(join(po + (at0 + h) * kD + 4 * lane, pe + at0 + h, step, pieces, 0, 1), row0 + h);
    }
}

template <typename T>
lf_status paged_t(const PagedArgs& a, const PagedPlan& pl, cudaStream_t stream) {
    lf_status st = LF_OK;
    if (pl.decode)
        st = launch_pdl(decode_kernel<T>, dim3((unsigned)a.n_seqs * pl.decode_splits, a.Hkv), dim3(kWarps * 32),
                        (size_t)pl.chunk * sizeof(int2), stream, a, pl);
    if (st == LF_OK && pl.tensor) st = launch_paged_tc(a, pl, stream);
    if (st != LF_OK || pl.splits() <= 1) return st;
    // A block per row for more than 16 pieces and no more blocks than run at
    // once (98 pieces of one context of 100000: 80 us by a warp per row, 23
    // by a block); eight heads a warp where there are more rows than half
    // warps (32768 rows of two pieces: 22 us by a warp per row).
    const long long rows = (long long)a.T * a.Hq;
    auto warps = [&](int each) { return dim3((unsigned)(((long long)a.T * ((a.Hq + each - 1) / each) + 7) / 8)); };
    if (pl.splits() > 16 && rows <= 8 * 148)
        return launch_pdl(merge_kernel<T, true, 1>, dim3((unsigned)rows), dim3(256), 0, stream, a, pl);
    if (rows <= 128 * 148) return launch_pdl(merge_kernel<T, false, 2>, warps(2), dim3(256), 0, stream, a, pl);
    return launch_pdl(merge_kernel<T, false, 8>, warps(8), dim3(256), 0, stream, a, pl);
}

}  // namespace

lf_status launch_paged_forward(const PagedArgs& a, const PagedPlan& pl, cudaStream_t stream) {
    return a.dtype == LF_F16 ? paged_t<__half>(a, pl, stream) : paged_t<__nv_bfloat16>(a, pl, stream);
}

}  // namespace lf
