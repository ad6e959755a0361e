// Windowed causal attention with sinks, forward, on the sm_100a tensor cores
// (fp16 / bf16): over packed or padded sequences, or over a paged cache.
//
// One CTA per tile of 128 query rows: 128 / G tokens times the G query heads
// that share a key/value head, so grouped heads read each key block once and
// a tile's keys span only w + 128 / G positions.  Per block of 64 keys:
//     S = Q K^T                        (tcgen05.mma, fp32 in tensor memory)
//     m' = max(m, max s), P = 2^(s - m'), l += sum P
//     O = O 2^(m - m') + P V           (P from tensor memory)
// Two threads share a row, each with its own half of every block's keys, its
// own m, l and O: they meet only at the tile's end, as two pieces of a split
// context would.  S has two buffers, so the next block's S runs under this
// one's softmax and the softmax warps never wait for a product; P overwrites
// the first 16 columns of its half of S.  S, S and two O's take 256 tensor-
// memory columns: two CTAs per SM.  (One thread a row, one S buffer and four
// CTAs per SM left every CTA a chain of latencies: 195 us at 16384 packed
// tokens, 16 / 4 heads, window 1024, 37 % of the issue slots used.)
// The O update is skipped unless a row's maximum grows by more than 2^8 (P
// <= 2^8 then).  P is rounded to the storage type, the MMA's operand type;
// sums stay fp32.
//
// Warps 0-7: softmax and epilogue, warp 8: TMA loads, warp 9: MMAs.  All
// waits are bounded (LF_ERR_DEVICE_TIMEOUT).
//
// Paged: a block is gathered by one TMA box per page (of up to 64
// positions).  Long contexts of few tiles are split over gridDim.z CTAs of
// `per` blocks each, which leave normalised fp32 rows and their log2-sum-exp
// for the merge kernel.
#include <atomic>
#include <mutex>

#include "lf_tc_tiles.cuh"

namespace lf {

namespace {
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}
}  // namespace

bool make_heads_map(CUtensorMap* m, const lf_heads& v, int heads, int tokens, int batches, int box_heads,
                    int box_tokens) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[4] = {64, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)batches};
    cuuint64_t strides[3] = {(cuuint64_t)v.head_stride * 2, (cuuint64_t)v.token_stride * 2,
                             (cuuint64_t)v.batch_stride * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, v.data, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

using namespace sm100;

constexpr int kBM = 128;   // query rows
constexpr int kBN = 64;    // keys per block
constexpr int kD = 64;
constexpr int kStages = 3;
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = (kSoftmaxWarps + 2) * 32;
constexpr int kCtas = 2;   // per SM
constexpr uint32_t kQBytes = kBM * kD * 2, kKBytes = kBN * kD * 2;
constexpr uint32_t kOffK = kQBytes, kOffV = kOffK + kStages * kKBytes, kOffMl = kOffV + kStages * kKBytes;
constexpr uint32_t kOffBar = kOffMl + 2 * kBM * 8;               // (m, l) of both halves
constexpr uint32_t kBars = 1 + 3 * kStages + 7;
constexpr uint32_t kOffMask = kOffBar + kBars * 8;               // valid keys of each stage (paged)
constexpr uint32_t kOffMisc = kOffMask + kStages * 8;
constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;            // + alignment slack
constexpr uint32_t kTmemCols = 256, kTmemO = 128;                // S at 0 and 64, O at 128 and 192
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;
static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "CTAs per SM");

struct Maps {
    CUtensorMap q, k, v;
};

template <typename T, bool kPaged, typename A>
__global__ void __launch_bounds__(kThreads, kCtas)
window_kernel(const __grid_constant__ Maps maps, const __grid_constant__ A a, const __grid_constant__ PagedPlan pl) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* k_full = q_full + 1;
    uint64_t* v_full = k_full + kStages;
    uint64_t* kv_empty = v_full + kStages;
    uint64_t* s_full = kv_empty + kStages;
    uint64_t* p_full = s_full + 2;  // (both [2]: per S buffer)
    uint64_t* pv_done = p_full + 2;
    uint64_t* o_full = pv_done + 1;
    uint64_t* drain = o_full + 1;
    float2* ml = reinterpret_cast<float2*>(smem + kOffMl);
    volatile unsigned long long* valid = reinterpret_cast<volatile unsigned long long*>(smem + kOffMask);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_launch_dependents();
    pdl_wait();
    const int G = a.Hq / a.Hkv, TQ = kBM / G, hk = blockIdx.y;
    int L;
    if constexpr (kPaged) L = a.T;
    else L = a.L;
    const int32_t* lens = nullptr;
    if constexpr (!kPaged) lens = a.lens;
    if (blockIdx.x == 0 && hk == 0 && blockIdx.z == 0) check_lengths(a.cu, lens, a.n_seqs, L, a.status);
    const TokenTile t = token_tile(a.cu, lens, a.n_seqs, L, TQ, blockIdx.x);
    if (t.t0 >= t.rows) return;
    int first = 0, n_keys = t.n;  // position of the first token, keys in all
    if constexpr (kPaged) {
        if (pl.decode && t.n * G <= kDecodeRows) return;  // the decode kernel's
        if (!paged_seq(a, t.b, t.n, n_keys, first, threadIdx.x == 0 && hk == 0 && blockIdx.z == 0 && t.t0 == 0)) return;
    }
    const int i0 = first + t.t0, i1 = first + imin(t.t0 + TQ, t.n) - 1;  // positions of the tile's tokens
    const KeyBlocks kb = tile_key_blocks(first, t.t0, imin(t.t0 + TQ, t.n), n_keys, a.w, a.sinks);
    int b0 = 0, b1 = kb.n;
    bool part = false;  // one piece of several
    if constexpr (kPaged) {
        b0 = imin(blockIdx.z * pl.per, kb.n);
        b1 = imin(b0 + pl.per, kb.n);
        part = kb.n > pl.per;
        if (b0 == b1 && blockIdx.z > 0) return;
    }
    const int nb = b1 - b0;

    // this thread's row and half (softmax warps)
    const int r = (warp & 3) * 32 + lane, half = warp >> 2, tok = t.t0 + r / G, head = hk * G + r % G;
    const bool row_stored = r < TQ * G && tok < t.rows;
    const size_t orow = ((size_t)t.batch * L + t.start + tok) * a.Hq + head;

    if (nb == 0) {  // padding, or nothing to see: zeros
        if (half > 0 || !row_stored) return;
        if constexpr (!kPaged) {
            a.lse[((size_t)t.batch * a.Hq + head) * L + t.start + tok] = -INFINITY;
        }
        zero_row64(static_cast<T*>(a.out) + orow * kD);
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&v_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(&p_full[0], kSoftmaxWarps);
        mbar_init(&p_full[1], kSoftmaxWarps);
        mbar_init(pv_done, 1);
        mbar_init(o_full, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kSoftmaxWarps + 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    if (warp == kSoftmaxWarps && lane == 0) {
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == kSoftmaxWarps) {
        // ------------------------------------------------------------ TMA
        bool ok = true;
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, (uint32_t)(TQ * G) * kD * 2);
            tma_load_4d(smem, &maps.q, q_full, 0, hk * G, t.start + t.t0, t.batch);
        }
        int j = 0;
        for (; j < nb; ++j) {
            const int s = j % kStages;
            ok = warp_wait(&kv_empty[s], ((j / kStages) & 1) ^ 1, abort_flag);
            if (!ok) break;
            const int c0 = key_block(kb, b0 + j) * kBN;
            uint8_t *ks = smem + kOffK + s * kKBytes, *vs = smem + kOffV + s * kKBytes;
            if constexpr (kPaged) {
                // lane u fetches the box of the block's u-th page
                const int shift = a.page_shift, rows = imin(kBN, 1 << shift), boxes = kBN / rows;
                const int pos = c0 + lane * rows;
                int page = -1;
                if (lane < boxes && pos < n_keys) {
                    page = page_of(a.table + (size_t)t.b * a.max_pages, a.max_pages, a.num_pages, shift, pos);
                    if (page < 0 && range_visible(imax(i0, 0), i1, pos, imin(pos + rows, n_keys) - 1, a.w, a.sinks))
                        record_status(a.status, t.b, LF_ERR_BAD_PAGE);
                }
                const unsigned have = __ballot_sync(0xffffffffu, page >= 0);
                if (lane == 0) {
                    unsigned long long m = 0;
                    for (int u = 0; u < boxes; ++u)
                        if ((have >> u) & 1) m |= low_bits64(rows) << (u * rows);
                    // and only keys some row sees: others' values may be anything
                    valid[s] = m & low_bits64(imin(n_keys, i1 + 1) - c0) &
                               (~low_bits64(imax(i0, 0) - a.w - c0) | low_bits64(a.sinks - c0));
                    const uint32_t bytes = __popc(have) * rows * kD * 2;
                    if (bytes) {
                        mbar_arrive_expect_tx(&k_full[s], bytes);
                        mbar_arrive_expect_tx(&v_full[s], bytes);
                    } else {
                        mbar_arrive(&k_full[s]);
                        mbar_arrive(&v_full[s]);
                    }
                }
                __syncwarp();
                if (page >= 0) {
                    const int slot = pos & ((1 << shift) - 1);
                    tma_load_4d(ks + lane * rows * kD * 2, &maps.k, &k_full[s], 0, hk, slot, page);
                    tma_load_4d(vs + lane * rows * kD * 2, &maps.v, &v_full[s], 0, hk, slot, page);
                }
                __syncwarp();
            } else if (lane == 0) {
                mbar_arrive_expect_tx(&k_full[s], kKBytes);
                tma_load_4d(ks, &maps.k, &k_full[s], 0, hk, t.start + c0, t.batch);
                mbar_arrive_expect_tx(&v_full[s], kKBytes);
                tma_load_4d(vs, &maps.v, &v_full[s], 0, hk, t.start + c0, t.batch);
            }
        }
        if (!ok && lane == 0) {  // wind-down: let issued copies land
            volatile int never = 0;
            mbar_wait(q_full, 0, &never, 200000000ull);
            for (int c = j > kStages ? j - kStages : 0; c < j; ++c) {
                mbar_wait(&k_full[c % kStages], (c / kStages) & 1, &never, 200000000ull);
                mbar_wait(&v_full[c % kStages], (c / kStages) & 1, &never, 200000000ull);
            }
        }
    } else if (warp == kSoftmaxWarps + 1) {
        // ------------------------------------------------------------ MMA
        // In issue order S_0, S_1, PV_0, S_2, PV_1, ...: the products run in
        // that order, so S_(j+1) may overwrite P_(j-1) without a wait.
        constexpr uint32_t id_s = idesc_f16(MmaFormat<T>::fmt, kBM, kBN, 0, 0);
        constexpr uint32_t id_o = idesc_f16(MmaFormat<T>::fmt, kBM, kD, 0, 1);
        const uint64_t dq = desc_sw128(smem_u32(smem)), dk = desc_sw128(smem_u32(smem + kOffK)),
                       dv = desc_sw128(smem_u32(smem + kOffV), 0);
        auto scores = [&](int j) -> bool {
            const int s = j % kStages;
            if (!warp_wait(&k_full[s], (j / kStages) & 1, abort_flag)) return false;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk)
                    mma_f16_ss(tmem + (j & 1) * kBN, dq + kk * 2, dk + s * (kKBytes >> 4) + kk * 2, id_s, kk > 0);
                tc_commit(&s_full[j & 1]);
            }
            __syncwarp();
            return true;
        };
        bool ok = warp_wait(q_full, 0, abort_flag) && scores(0);
        for (int j = 0; j < nb && ok; ++j) {
            const int s = j % kStages;
            // S_(j+1) reuses the buffer of P_(j-1): its PV has been issued
            if (j + 1 < nb) ok = scores(j + 1);
            ok = ok && warp_wait(&v_full[s], (j / kStages) & 1, abort_flag) &&
                 warp_wait(&p_full[j & 1], (j >> 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)  // two steps of 16 keys for each half's O
                    mma_f16_ts(tmem + kTmemO + (kk >> 1) * kD, tmem + (j & 1) * kBN + (kk >> 1) * 32 + (kk & 1) * 8,
                               dv + s * (kKBytes >> 4) + kk * (2048 >> 4), id_o, j > 0 || (kk & 1));
                tc_commit(&kv_empty[s]);
                tc_commit(pv_done);
                if (j == nb - 1) tc_commit(o_full);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) {  // wind-down: wait for the MMAs already issued
            volatile int never = 0;
            tc_commit(drain);
            mbar_wait(drain, 0, &never, 200000000ull);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tO = t_lane + kTmemO + half * kD;
        const int i = r < TQ * G && tok < t.n ? first + tok : -1;
        const float sc = a.scale * kLog2e;
        // blocks that every row sees whole begin in [full_lo, full_hi]
        const int full_lo = i1 - a.w, full_hi = imin(i0 + 1, n_keys) - kBN;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < nb; ++j) {
            const int s = j % kStages, c0 = key_block(kb, b0 + j) * kBN;
            const uint32_t tS = t_lane + (j & 1) * kBN + half * 32;
            bool full = c0 <= full_hi && c0 >= full_lo;
            ok = warp_wait(&s_full[j & 1], (j >> 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            float x[32];
            tmem_ld32f(tS, x);
            unsigned long long have = ~0ull;  // keys that exist (and, paged, that some row sees)
            if constexpr (kPaged) {
                // (published before the loads of the stage were issued)
                ok = warp_wait(&k_full[s], (j / kStages) & 1, abort_flag);
                if (!ok) break;
                have = valid[s];
                full = full && have == ~0ull;
            } else if (c0 + kBN > n_keys) {
                have = low_bits64(n_keys - c0);
            }
            tmem_ld_wait();
            regs_ready<32>(x);
            if (!full) {
                const uint32_t bits = visible_bits32(i, c0 + half * 32, n_keys, a.w, a.sinks) & (uint32_t)(have >> (32 * half));
#pragma unroll
                for (int c = 0; c < 32; ++c) x[c] = (bits >> c) & 1 ? x[c] : -INFINITY;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
                mx[0] = max3(mx[0], x[c], x[c + 1]);
                mx[1] = max3(mx[1], x[c + 2], x[c + 3]);
                mx[2] = max3(mx[2], x[c + 4], x[c + 5]);
                mx[3] = max3(mx[3], x[c + 6], x[c + 7]);
            }
            const float cm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
            const bool need = cm > m + kRescale || (m == -INFINITY && cm > m);
            if (__any_sync(0xffffffffu, need)) {
                const bool real = need && m != -INFINITY;
                if (__any_sync(0xffffffffu, real)) {
                    // every earlier product into O must be done (PV_(j-2) and
                    // before are, since S_j is)
                    ok = warp_wait(pv_done, (j - 1) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const float f = real ? ex2(m - cm) : 1.0f;
                    l *= f;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        float o[16];
                        tmem_ld16f(tO + h * 16, o);
                        tmem_ld_wait();
                        regs_ready<16>(o);
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] *= f;
                        tmem_st16f(tO + h * 16, o);
                    }
                }
                if (need) m = cm;
            }
            const float nm = m == -INFINITY ? 0.0f : -m;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float e0 = ex2(fmaf(x[2 * c], sc, nm)), e1 = ex2(fmaf(x[2 * c + 1], sc, nm));
                sum[(2 * c) & 3] += e0;
                sum[(2 * c + 1) & 3] += e1;
                pk[c] = Pair<T>::pack(e0, e1);
            }
            tmem_st16(tS, pk);
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (have != ~0ull) {
                // rows of V that are no key of the sequence: 0 * NaN is NaN
                ok = warp_wait(&v_full[s], (j / kStages) & 1, abort_flag);
                if (!ok) break;
                const int row = threadIdx.x >> 2;
                if (!((have >> row) & 1)) {
                    uint4* z = reinterpret_cast<uint4*>(smem + kOffV + s * kKBytes + row * 128 + (threadIdx.x & 3) * 32);
                    z[0] = z[1] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[j & 1]);
        }
        if (ok) ok = warp_wait(o_full, 0, abort_flag);
        // join the halves (an abort is seen by all eight warps or comes too
        // late to matter: the barrier below is reached either way)
        ml[half * kBM + r] = make_float2(m, l);
        named_bar_sync(1, kSoftmaxWarps * 32);
        if (ok) {
            tc_fence_after();
            const float2 u0 = ml[r], u1 = ml[kBM + r];
            const float top = fmaxf(u0.x, u1.x), base = top == -INFINITY ? 0.0f : top;
            const float f0 = ex2(u0.x - base), f1 = ex2(u1.x - base);
            const float sum = i >= 0 ? u0.y * f0 + u1.y * f1 : 0.0f;  // i < 0: no token of the sequence
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const float lse2 = sum == 0.0f ? -INFINITY : top + log2f(sum);
            const size_t at = part ? (size_t)blockIdx.z * ((size_t)L * a.Hq) + orow : 0;
            float o[32], o1[32];
            tmem_ld32f(t_lane + kTmemO + half * 32, o);
            tmem_ld32f(t_lane + kTmemO + kD + half * 32, o1);
            tmem_ld_wait();
            regs_ready<32>(o);
            regs_ready<32>(o1);
            // (a half that saw no key holds exact zeros)
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = sum == 0.0f ? 0.0f : o[c] * f0 + o1[c] * f1;
            if (row_stored) {
                if (part) {
                    float4* d = reinterpret_cast<float4*>(pl.o + at * kD + half * 32);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        d[c] = make_float4(o[4 * c] * inv, o[4 * c + 1] * inv, o[4 * c + 2] * inv, o[4 * c + 3] * inv);
                    if (half == 0) pl.lse[at] = lse2;
                } else {
                    store_row32(static_cast<T*>(a.out) + orow * kD + half * 32, o, inv);
                    if constexpr (!kPaged) {
                        if (half == 0) a.lse[((size_t)t.batch * a.Hq + head) * L + t.start + tok] = lse2 * kLn2;
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) record_status(a.status, 0, LF_ERR_DEVICE_TIMEOUT);
    if (warp == kSoftmaxWarps + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <typename T, bool kPaged, typename A>
lf_status launch(const Maps& maps, const A& a, const PagedPlan& pl, dim3 grid, cudaStream_t stream) {
    static std::atomic<bool> attr[64];  // the shared-memory opt-in, per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return LF_ERR_CUDA;
    if (!attr[dev].load()) {
        if (cudaFuncSetAttribute(window_kernel<T, kPaged, A>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemBytes) != cudaSuccess)
            return LF_ERR_CUDA;
        attr[dev].store(true);
    }
    return launch_pdl(window_kernel<T, kPaged, A>, grid, dim3(kThreads), kSmemBytes, stream, maps, a, pl);
}

}  // namespace

lf_status launch_window_forward_tc(const WindowArgs& a, cudaStream_t stream) {
    const int G = a.heads_group(), TQ = kBM / G, B = a.packed() ? 1 : a.n_seqs;
    Maps maps;
    if (!make_heads_map(&maps.q, a.q, a.Hq, a.L, B, G, TQ) || !make_heads_map(&maps.k, a.k, a.Hkv, a.L, B, 1, kBN) ||
        !make_heads_map(&maps.v, a.v, a.Hkv, a.L, B, 1, kBN))
        return LF_ERR_CUDA;
    const dim3 grid(token_slots(a.packed(), a.n_seqs, a.L, TQ), a.Hkv);
    const PagedPlan pl = {};
    if (a.dtype == LF_F16) return launch<__half, false>(maps, a, pl, grid, stream);
    return launch<__nv_bfloat16, false>(maps, a, pl, grid, stream);
}

lf_status launch_paged_tc(const PagedArgs& a, const PagedPlan& pl, cudaStream_t stream) {
    const int G = a.heads_group(), TQ = kBM / G, page = 1 << a.page_shift;
    Maps maps;
    if (!make_heads_map(&maps.q, a.q, a.Hq, a.T, 1, G, TQ) ||
        !make_heads_map(&maps.k, a.k, a.Hkv, page, a.num_pages, 1, imin(page, kBN)) ||
        !make_heads_map(&maps.v, a.v, a.Hkv, page, a.num_pages, 1, imin(page, kBN)))
        return LF_ERR_CUDA;
    const dim3 grid(packed_slots(a.T, a.n_seqs, TQ), a.Hkv, pl.tensor_splits);
    if (a.dtype == LF_F16) return launch<__half, true>(maps, a, pl, grid, stream);
    return launch<__nv_bfloat16, true>(maps, a, pl, grid, stream);
}

}  // namespace lf
