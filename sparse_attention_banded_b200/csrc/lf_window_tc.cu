// Windowed causal attention with sinks, forward, on the sm_100a tensor cores
// (fp16 / bf16): over packed or padded sequences, or over a paged cache.
//
// A persistent CTA works on tiles of 128 query rows: 128 / G tokens times the
// G query heads that share a key/value head, so grouped heads read each key
// block once and a tile's keys span only w + 128 / G positions.  Per block of
// 64 keys:
//     S = Q K^T                        (tcgen05.mma, fp32 in tensor memory)
//     m' = max(m, max s), P = 2^(s - m'), l += sum P
//     O = O 2^(m - m') + P V           (P from tensor memory)
// One thread per row; P overwrites the first half of S's columns.  A CTA's
// block is a chain of latencies (product, softmax, product: 2500 cycles, of
// which the arithmetic is a third).  Many tiles: S and O take 128
// tensor-memory columns, four CTAs per SM, and their chains fill each other's
// gaps.  (4 x 4096 tokens, 16 heads, window 256: 59 us, and 70 with two CTAs
// per SM and two threads a row.)  Few tiles: two CTAs per SM with two buffers
// of S, and the next block's S runs under this one's softmax (two chunks of
// 1024 tokens, 16 / 4 heads, window 4096, 264 items: 78 us with the append,
// and 104 the other way).
// A tile of its own launch paid 8000 cycles more to start and end, so CTAs
// are persistent and the loads and plan of the next tile run under the end of
// this one.  The four softmax warps keep 64 scores a row in registers, of the
// share that the other warps give up.
// The O update is skipped unless a row's maximum grows by more than 2^8 (P
// <= 2^8 then).  P is rounded to the storage type, the MMA's operand type;
// sums stay fp32.
//
// Warps 0-3: softmax and epilogue, warp 4: TMA loads, warp 5: MMAs, warp 6:
// the plans of the coming tiles (which sequence, which keys).  All waits are
// bounded (LF_ERR_DEVICE_TIMEOUT).
//
// Paged: a block is gathered by one TMA box per page (of up to 64
// positions).  Long contexts of few tiles are split into items of `per`
// blocks each, which leave normalised fp32 rows and their log2-sum-exp
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
constexpr int kRing = 4;   // plans ahead
constexpr int kSoftmaxWarps = 4;
constexpr int kTmaWarp = 4, kMmaWarp = 5, kPlanWarp = 6;
constexpr int kThreads = 8 * 32;
constexpr uint32_t kQBytes = kBM * kD * 2, kKBytes = kBN * kD * 2;
constexpr uint32_t kPlanBytes = 80;

// The two ways a CTA is laid out (the rule: kAheadItems).
//   kAhead false: four CTAs per SM, each a chain of S, softmax, P V.
//   kAhead true: two CTAs per SM, S double-buffered: the next block's S runs
//   under this one's softmax, which shortens the chain of a lone CTA.
template <bool kAhead>
struct Layout {
    static constexpr int kCtas = kAhead ? 2 : 4;  // per SM
    static constexpr int kStages = kAhead ? 4 : 2;
    static constexpr int kBufs = kAhead ? 2 : 1;  // of S
    // Registers a thread at launch; a block's share is split anew.  (Four
    // CTAs, the padded batch: 24 and 104 59 us, 32 and 96 60, 40 and 88 66.)
    // Code of warps 4 to 7 must stay inline: after they have given registers
    // away, a call out of line (a device printf, a 64-bit division, a helper
    // that is not inlined) may use more than the warp has left, which is an
    // illegal instruction.  ptxas keeps what is inlined to the share; four
    // CTAs of the paged form spill 224 and 368 bytes for it, the other 80 and
    // 92.
    static constexpr uint32_t kRegsLaunch = kAhead ? 128 : 64, kRegsProducer = kAhead ? 96 : 24,
                              kRegsSoftmax = kAhead ? 160 : 104;
    static_assert(4 * 32 * kRegsProducer + 4 * 32 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");
    static constexpr uint32_t kOffK = kQBytes, kOffV = kOffK + kStages * kKBytes, kOffPlan = kOffV + kStages * kKBytes;
    static constexpr uint32_t kOffBar = kOffPlan + kRing * kPlanBytes;
    static constexpr uint32_t kBars = 2 + 2 * kStages + 2 * kBufs + 2 + 2 * kRing;
    static constexpr uint32_t kOffMask = kOffBar + kBars * 8;  // valid keys of each stage (paged)
    static constexpr uint32_t kOffMisc = kOffMask + kStages * 8;
    static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;  // + alignment slack
    static constexpr uint32_t kTmemCols = kAhead ? 256 : 128, kTmemO = kBufs * kBN;  // S (then P) before O
    static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "CTAs per SM");
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;

struct Maps {
    CUtensorMap q, k, v;
};

// What a tile's roles need to know; nb = 0: rows of zeros (padding, or
// nothing to see), nb < 0: no more tiles.
struct Plan {
    int nb, b0, n_sink, lo;    // blocks [b0, b0 + nb) of the list n_sink, lo
    int i0, i1, n_keys;        // positions of its tokens, keys of the sequence
    int first;                 // position of the sequence's first token
    int b, batch, start, t0;   // sequence, its batch and first row; the tile's first token
    int n, rows, hk;           // tokens, stored rows of the sequence; key/value head
    int part, z;               // one piece of several: index
    __device__ __forceinline__ int key0(int j) const {  // first key of the tile's j-th block
        j += b0;
        return (j < n_sink ? j : lo + (j - n_sink)) * kBN;
    }
};
static_assert(sizeof(Plan) <= kPlanBytes, "plan slot");

template <bool kPaged, typename A>
__device__ __forceinline__ int rows_total(const A& a) {
    if constexpr (kPaged) return a.T;
    else return a.L;
}

// The plan of an item; false: the item has no work at all.
template <bool kPaged, typename A>
__device__ bool make_plan(const A& a, const PagedPlan& pp, int item, Plan& p, bool report) {
    const int G = a.Hq / a.Hkv, TQ = kBM / G;
    int slot = item, z = 0;
    if constexpr (kPaged) {
        z = slot % pp.tensor_splits;
        slot /= pp.tensor_splits;
    }
    p.hk = slot % a.Hkv;
    slot /= a.Hkv;
    const int32_t* lens = nullptr;
    if constexpr (!kPaged) lens = a.lens;
    const TokenTile t = token_tile(a.cu, lens, a.n_seqs, rows_total<kPaged>(a), TQ, slot);
    if (t.t0 >= t.rows) return false;
    p.first = 0;
    p.n_keys = t.n;
    if constexpr (kPaged) {
        if (pp.decode && t.n * G <= kDecodeRows) return false;  // the decode kernel's
        if (!paged_seq(a, t.b, t.n, p.n_keys, p.first, report && p.hk == 0 && z == 0 && t.t0 == 0)) return false;
    }
    const int t1 = imin(t.t0 + TQ, t.n);
    const KeyBlocks kb = tile_key_blocks(p.first, t.t0, t1, p.n_keys, a.w, a.sinks);
    p.i0 = p.first + t.t0;
    p.i1 = p.first + t1 - 1;
    p.n_sink = kb.n_sink;
    p.lo = kb.lo;
    p.b0 = 0;
    p.nb = kb.n;
    p.part = 0;
    p.z = z;
    if constexpr (kPaged) {
        p.b0 = imin(z * pp.per, kb.n);
        p.nb = imin(p.b0 + pp.per, kb.n) - p.b0;
        p.part = kb.n > pp.per;
        if (p.nb == 0 && z > 0) return false;
    }
    p.b = t.b;
    p.batch = t.batch;
    p.start = t.start;
    p.t0 = t.t0;
    p.n = t.n;
    p.rows = t.rows;
    return true;
}

template <typename T, bool kPaged, bool kAhead, typename A>
__global__ void __launch_bounds__(kThreads, Layout<kAhead>::kCtas)
window_kernel(const __grid_constant__ Maps maps, const __grid_constant__ A a, const __grid_constant__ PagedPlan pp,
              int n_items) {
    using Lay = Layout<kAhead>;
    constexpr int kStages = Lay::kStages, kBufs = Lay::kBufs;
    constexpr uint32_t kOffK = Lay::kOffK, kOffV = Lay::kOffV, kOffPlan = Lay::kOffPlan, kTmemO = Lay::kTmemO;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Lay::kOffBar);
    uint64_t* q_empty = q_full + 1;
    uint64_t* kv_full = q_empty + 1;
    uint64_t* kv_empty = kv_full + kStages;
    uint64_t* s_full = kv_empty + kStages;  // [kBufs], as the next
    uint64_t* p_full = s_full + kBufs;
    uint64_t* o_full = p_full + kBufs;
    uint64_t* drain = o_full + 1;
    uint64_t* plan_full = drain + 1;
    uint64_t* plan_empty = plan_full + kRing;
    volatile uint32_t* valid = reinterpret_cast<volatile uint32_t*>(smem + Lay::kOffMask);  // [stage][2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::kOffMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int u = 0; u < kBufs; ++u) {
            mbar_init(&s_full[u], 1);
            mbar_init(&p_full[u], kSoftmaxWarps);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        mbar_init(o_full, 1);
        mbar_init(drain, 1);
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&plan_full[s], 1);
            mbar_init(&plan_empty[s], kSoftmaxWarps + 2);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kTmaWarp && lane == 0) {
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    // (only now: a kernel that runs before may hold tensor memory until it ends)
    pdl_wait();
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, Lay::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const int G = a.Hq / a.Hkv, TQ = kBM / G, L = rows_total<kPaged>(a);

    // The plans, in order; the slot of plan k - 1 is handed back when the
    // role asks for plan k.  NULL after an abort.
    auto next_plan = [&](int k) -> const Plan* {
        if (k > 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&plan_empty[(k - 1) % kRing]);
        }
        if (!warp_wait(&plan_full[k % kRing], (k / kRing) & 1, abort_flag)) return nullptr;
        return reinterpret_cast<const Plan*>(smem + kOffPlan + (k % kRing) * kPlanBytes);
    };

    if (warp >= kSoftmaxWarps) {
        regs_dec<Lay::kRegsProducer>();
        if (warp == kPlanWarp) {
            // -------------------------------------------------------- plans
            const int32_t* lens = nullptr;
            if constexpr (!kPaged) lens = a.lens;
            if (blockIdx.x == 0) check_lengths(a.cu, lens, a.n_seqs, L, a.status, lane, 32);
            int k = 0;
            for (int item = blockIdx.x;; item += gridDim.x) {
                Plan p;
                p.nb = -1;
                if (item < n_items && !make_plan<kPaged>(a, pp, item, p, lane == 0)) continue;
                if (!warp_wait(&plan_empty[k % kRing], ((k / kRing) & 1) ^ 1, abort_flag)) break;
                if (lane == 0) {
                    *reinterpret_cast<Plan*>(smem + kOffPlan + (k % kRing) * kPlanBytes) = p;
                    mbar_arrive(&plan_full[k % kRing]);
                }
                ++k;
                if (p.nb < 0) break;
            }
        } else if (warp == kTmaWarp) {
            // -------------------------------------------------------- TMA
            bool ok = true;
            int g = 0, it = 0;  // blocks, tiles with blocks so far
            for (int k = 0; ok; ++k) {
                const Plan* p = next_plan(k);
                if (!p || p->nb < 0) {
                    ok = p != nullptr;
                    break;
                }
                if (p->nb == 0) continue;
                ok = warp_wait(q_empty, (it & 1) ^ 1, abort_flag);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, (uint32_t)(TQ * G) * kD * 2);
                    tma_load_4d(smem, &maps.q, q_full, 0, p->hk * G, p->start + p->t0, p->batch);
                }
                ++it;
                const int hk = p->hk, n_keys = p->n_keys, nb = p->nb;
                // Paged: a lane looks up the page of one box, those of 32 /
                // boxes blocks at a time and as many ahead.
                [[maybe_unused]] int next_page = -1, next_pos = 0, page = -1, pos = 0, rows = 0, boxes = 1;
                [[maybe_unused]] auto look_up = [&](int j) {
                    if constexpr (kPaged) {
                        j += lane / boxes;
                        next_page = -1;
                        if (j < nb) {
                            next_pos = p->key0(j) + lane % boxes * rows;
                            if (next_pos < n_keys) {
                                next_page = page_of(a.table + (size_t)p->b * a.max_pages, a.max_pages, a.num_pages,
                                                    a.page_shift, next_pos);
                                if (next_page < 0 && range_visible(imax(p->i0, 0), p->i1, next_pos,
                                                                   imin(next_pos + rows, n_keys) - 1, a.w, a.sinks))
                                    record_status(a.status, p->b, LF_ERR_BAD_PAGE);
                            }
                        }
                    }
                };
                if constexpr (kPaged) {
                    rows = imin(kBN, 1 << a.page_shift);
                    boxes = kBN / rows;
                    look_up(0);
                }
                for (int j = 0; j < nb; ++j, ++g) {
                    const int s = g % kStages;
                    const int c0 = p->key0(j);
                    uint8_t *ks = smem + kOffK + s * kKBytes, *vs = smem + kOffV + s * kKBytes;
                    if constexpr (kPaged) {
                        const int first_lane = j % (32 / boxes) * boxes, box = lane - first_lane;
                        if (first_lane == 0) {
                            page = next_page;
                            pos = next_pos;
                            look_up(j + 32 / boxes);
                        }
                        const bool mine = box >= 0 && box < boxes && page >= 0;
                        const unsigned have = __ballot_sync(0xffffffffu, mine) >> first_lane;
                        ok = warp_wait(&kv_empty[s], ((g / kStages) & 1) ^ 1, abort_flag);
                        if (!ok) break;
                        if (lane == 0) {
                            unsigned long long m = 0;
                            for (int u = 0; u < boxes; ++u)
                                if ((have >> u) & 1) m |= low_bits64(rows) << (u * rows);
                            // and only keys some row sees: others' values may be anything
                            m &= low_bits64(imin(n_keys, p->i1 + 1) - c0) &
                                 (~low_bits64(imax(p->i0, 0) - a.w - c0) | low_bits64(a.sinks - c0));
                            valid[2 * s] = (uint32_t)m;
                            valid[2 * s + 1] = (uint32_t)(m >> 32);
                            const uint32_t bytes = __popc(have) * rows * kD * 2;
                            if (bytes) mbar_arrive_expect_tx(&kv_full[s], 2 * bytes);
                            else mbar_arrive(&kv_full[s]);
                        }
                        __syncwarp();
                        if (mine) {
                            const int slot = pos & ((1 << a.page_shift) - 1);
                            tma_load_4d(ks + box * rows * kD * 2, &maps.k, &kv_full[s], 0, hk, slot, page);
                            tma_load_4d(vs + box * rows * kD * 2, &maps.v, &kv_full[s], 0, hk, slot, page);
                        }
                        __syncwarp();
                    } else {
                        ok = warp_wait(&kv_empty[s], ((g / kStages) & 1) ^ 1, abort_flag);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&kv_full[s], 2 * kKBytes);
                            tma_load_4d(ks, &maps.k, &kv_full[s], 0, hk, p->start + c0, p->batch);
                            tma_load_4d(vs, &maps.v, &kv_full[s], 0, hk, p->start + c0, p->batch);
                        }
                        __syncwarp();
                    }
                }
            }
            if (!ok && lane == 0) {  // wind-down: let issued copies land
                volatile int never = 0;
                if (it > 0) mbar_wait(q_full, (it - 1) & 1, &never, 200000000ull);
                for (int c = g > kStages ? g - kStages : 0; c < g; ++c)
                    mbar_wait(&kv_full[c % kStages], (c / kStages) & 1, &never, 200000000ull);
            }
        } else if (warp == kMmaWarp) {
            // -------------------------------------------------------- MMA
            // In issue order S_0, PV_0, S_1, PV_1, ... (or, ahead, S_0, S_1,
            // PV_0, S_2, PV_1, ...): the products run in that order, so S of
            // a block may overwrite P of the last one in its buffer without a
            // wait.  The first PV of a tile overwrites O: it waits for the P
            // of warps that have read the last tile's O.
            constexpr uint32_t id_s = idesc_f16(MmaFormat<T>::fmt, kBM, kBN, 0, 0);
            constexpr uint32_t id_o = idesc_f16(MmaFormat<T>::fmt, kBM, kD, 0, 1);
            const uint64_t dq = desc_sw128(smem_u32(smem)), dk = desc_sw128(smem_u32(smem + kOffK)),
                           dv = desc_sw128(smem_u32(smem + kOffV), 0);
            bool ok = true;
            int g = 0, it = 0;
            for (int k = 0; ok; ++k) {
                const Plan* p = next_plan(k);
                if (!p || p->nb < 0) {
                    ok = p != nullptr;
                    break;
                }
                const int nb = p->nb;
                if (nb == 0) continue;
                auto scores = [&](int j) -> bool {
                    const int c = g + j, s = c % kStages;
                    if (!warp_wait(&kv_full[s], (c / kStages) & 1, abort_flag)) return false;
                    tc_fence_after();
                    mma4_ss(tmem + c % kBufs * kBN, dq, dk + s * (kKBytes >> 4), id_s);
                    commit_elect(&s_full[c % kBufs]);
                    if (j == nb - 1) commit_elect(q_empty);
                    return true;
                };
                ok = warp_wait(q_full, it & 1, abort_flag);
                if (kAhead) ok = ok && scores(0);
                for (int j = 0; j < nb && ok; ++j) {
                    const int c = g + j, s = c % kStages;
                    if (!kAhead) ok = scores(j);
                    else if (j + 1 < nb) ok = scores(j + 1);
                    ok = ok && warp_wait(&p_full[c % kBufs], (c / kBufs) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    mma4_ts<16>(tmem + kTmemO, tmem + kTmemO, tmem + c % kBufs * kBN, dv + s * (kKBytes >> 4), id_o,
                                j > 0, 1);
                    commit_elect(&kv_empty[s]);
                    if (j == nb - 1) commit_elect(o_full);
                }
                g += nb;
                ++it;
            }
            if (!ok) {  // wind-down: wait for the MMAs already issued
                volatile int never = 0;
                commit_elect(drain);
                mbar_wait(drain, 0, &never, 200000000ull);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        regs_inc<Lay::kRegsSoftmax>();
        // this thread's row of a tile
        const int r = threadIdx.x;
        const int r_tok = r / G, r_head = r % G;
        const bool row_used = r < TQ * G;
        const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16), tO = t_lane + kTmemO;
        const float sc = a.scale * kLog2e;
        bool ok = true;
        int g = 0, it = 0;
        for (int k = 0; ok; ++k) {
            const Plan* p = next_plan(k);
            if (!p || p->nb < 0) break;
            const int nb = p->nb, n_keys = p->n_keys, tok = p->t0 + r_tok;
            const bool row_stored = row_used && tok < p->rows;
            const int i = row_used && tok < p->n ? p->first + tok : -1;  // this row's position
            if (nb == 0) {
                if (row_stored) {
                    const size_t orow = ((size_t)p->batch * L + p->start + tok) * a.Hq + p->hk * G + r_head;
                    zero_row64(static_cast<T*>(a.out) + orow * kD);
                    if constexpr (!kPaged)
                        a.lse[((size_t)p->batch * a.Hq + p->hk * G + r_head) * L + p->start + tok] = -INFINITY;
                }
                continue;
            }
            // blocks that every row sees whole begin in [full_lo, full_hi]
            const int full_lo = p->i1 - a.w, full_hi = imin(p->i0 + 1, n_keys) - kBN;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < nb; ++j) {
                const int c = g + j, s = c % kStages, c0 = p->key0(j);
                const uint32_t tS = t_lane + c % kBufs * kBN;
                bool full = c0 <= full_hi && c0 >= full_lo;
                ok = warp_wait(&s_full[c % kBufs], (c / kBufs) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                float x[kBN];
                tmem_ld32f(tS, x);
                tmem_ld32f(tS + 32, x + 32);
                bool all = c0 + kBN <= n_keys;  // every key exists (and, paged, some row sees it)
                if constexpr (kPaged) {
                    // (published before the loads of the stage were issued)
                    ok = warp_wait(&kv_full[s], (c / kStages) & 1, abort_flag);
                    if (!ok) break;
                    all = valid[2 * s] == ~0u && valid[2 * s + 1] == ~0u;
                    full = full && all;
                }
                auto have = [&](int h) -> uint32_t {
                    if constexpr (kPaged) return valid[2 * s + h];
                    else return low_bits32(n_keys - c0 - 32 * h);
                };
                tmem_ld_wait();
                regs_ready<kBN>(x);
                if (!full) {
                    const uint32_t lo = visible_bits32(i, c0, n_keys, a.w, a.sinks) & have(0);
                    const uint32_t hi = visible_bits32(i, c0 + 32, n_keys, a.w, a.sinks) & have(1);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        x[e] = (lo >> e) & 1 ? x[e] : -INFINITY;
                        x[e + 32] = (hi >> e) & 1 ? x[e + 32] : -INFINITY;
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < kBN; e += 8) {
                    mx[0] = max3(mx[0], x[e], x[e + 1]);
                    mx[1] = max3(mx[1], x[e + 2], x[e + 3]);
                    mx[2] = max3(mx[2], x[e + 4], x[e + 5]);
                    mx[3] = max3(mx[3], x[e + 6], x[e + 7]);
                }
                const float cm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                const bool need = cm > m + kRescale || (m == -INFINITY && cm > m);
                float f = 1.0f;
                bool real = false;
                if (need) {
                    real = m != -INFINITY;
                    f = real ? ex2(m - cm) : 1.0f;
                    m = cm;
                    l *= f;
                }
                const float nm = m == -INFINITY ? 0.0f : -m;
                const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(nm, nm);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 v = ffma2(make_float2(x[32 * h + 2 * e], x[32 * h + 2 * e + 1]), sc2, nm2);
                        const float2 q = make_float2(ex2(v.x), ex2(v.y));
                        sum[e & 1] = fadd2(sum[e & 1], q);
                        pk[e] = Pair<T>::pack(q.x, q.y);
                    }
                    tmem_st16(tS + h * 16, pk);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                if (__any_sync(0xffffffffu, real)) {
                    // The products into O must be done.  They are, since S of
                    // this block is, but for the last one where S runs ahead:
                    // it releases its stage (and none follows without this
                    // warp's P).
                    if (kAhead) {
                        ok = warp_wait(&kv_empty[(c - 1) % kStages], ((c - 1) / kStages) & 1, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        float o[16];
                        tmem_ld16f(tO + h * 16, o);
                        tmem_ld_wait();
                        regs_ready<16>(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= f;
                        tmem_st16f(tO + h * 16, o);
                    }
                }
                if (!all) {
                    // rows of V that are no key of the sequence: 0 * NaN is NaN
                    ok = warp_wait(&kv_full[s], (c / kStages) & 1, abort_flag);
                    if (!ok) break;
                    const int row = threadIdx.x >> 1;
                    if (!((have(row >> 5) >> (row & 31)) & 1)) {
                        uint4* zr = reinterpret_cast<uint4*>(smem + kOffV + s * kKBytes + row * 128 + (threadIdx.x & 1) * 64);
#pragma unroll
                        for (int u = 0; u < 4; ++u) zr[u] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[c % kBufs]);
            }
            if (ok) ok = warp_wait(o_full, it & 1, abort_flag);
            if (ok) {
                tc_fence_after();
                const bool none = i < 0 || l == 0.0f;  // no token of the sequence, or no key
                const float inv = rcp_approx(l), lse2 = none ? -INFINITY : m + lg2_approx(l);
                const size_t orow = ((size_t)p->batch * L + p->start + tok) * a.Hq + p->hk * G + r_head;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float o[32];
                    tmem_ld32f(tO + h * 32, o);
                    tmem_ld_wait();
                    regs_ready<32>(o);
                    if (h == 1) tc_fence_before();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] *= inv;
                    if (none) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.0f;
                    }
                    if (row_stored) {
                        if (kPaged && p->part) {
                            float4* d = reinterpret_cast<float4*>(pp.o(a.Hq) + ((size_t)p->z * ((size_t)L * a.Hq) + orow) * kD + h * 32);
#pragma unroll
                            for (int e = 0; e < 8; ++e) d[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        } else {
                            store_row32(static_cast<T*>(a.out) + orow * kD + h * 32, o);
                        }
                    }
                    __syncwarp();
                }
                if (row_stored) {
                    if (kPaged && p->part) pp.lse(L, a.Hq)[(size_t)p->z * ((size_t)L * a.Hq) + orow] = lse2;
                    if constexpr (!kPaged)
                        a.lse[((size_t)p->batch * a.Hq + p->hk * G + r_head) * L + p->start + tok] = lse2 * kLn2;
                }
                __syncwarp();
            }
            g += nb;
            ++it;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) record_status(a.status, 0, LF_ERR_DEVICE_TIMEOUT);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, Lay::kTmemCols);
    }
}

template <typename T, bool kPaged, bool kAhead, typename A>
lf_status launch_as(const Maps& maps, const A& a, const PagedPlan& pp, int items, DeviceCtx* d, cudaStream_t stream) {
    static std::atomic<bool> attr[64];  // the shared-memory opt-in, per device
    using Lay = Layout<kAhead>;
    if (!attr[d->ordinal].load()) {
        if (cudaFuncSetAttribute(window_kernel<T, kPaged, kAhead, A>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Lay::kSmemBytes) != cudaSuccess)
            return LF_ERR_CUDA;
        attr[d->ordinal].store(true);
    }
    const int grid = imin(items, Lay::kCtas * d->sm_count);
    return launch_pdl(window_kernel<T, kPaged, kAhead, A>, dim3(grid), dim3(kThreads), Lay::kSmemBytes, stream, maps, a, pp,
                      items);
}

template <typename T, bool kPaged, typename A>
lf_status launch(const Maps& maps, const A& a, const PagedPlan& pp, long long items, bool ahead, cudaStream_t stream) {
    lf_status st;
    DeviceCtx* d = current_device(&st);
    if (!d) return st;
    if (items > kMostItems) return LF_ERR_TOO_LARGE;
    return ahead ? launch_as<T, kPaged, true>(maps, a, pp, (int)items, d, stream)
                 : launch_as<T, kPaged, false>(maps, a, pp, (int)items, d, stream);
}

}  // namespace

lf_status launch_window_forward_tc(const WindowArgs& a, cudaStream_t stream) {
    const int G = a.heads_group(), TQ = kBM / G, B = a.packed() ? 1 : a.n_seqs;
    Maps maps;
    if (!make_heads_map(&maps.q, a.q, a.Hq, a.L, B, G, TQ) || !make_heads_map(&maps.k, a.k, a.Hkv, a.L, B, 1, kBN) ||
        !make_heads_map(&maps.v, a.v, a.Hkv, a.L, B, 1, kBN))
        return LF_ERR_CUDA;
    const PagedPlan pp = {};
    const long long items = (long long)token_slots(a.packed(), a.n_seqs, a.L, TQ) * a.Hkv;
    const bool ahead = items <= kAheadItems;
    if (a.dtype == LF_F16) return launch<__half, false>(maps, a, pp, items, ahead, stream);
    return launch<__nv_bfloat16, false>(maps, a, pp, items, ahead, stream);
}

lf_status launch_paged_tc(const PagedArgs& a, const PagedPlan& pp, cudaStream_t stream) {
    const int G = a.heads_group(), TQ = kBM / G, page = 1 << a.page_shift;
    Maps maps;
    if (!make_heads_map(&maps.q, a.q, a.Hq, a.T, 1, G, TQ) ||
        !make_heads_map(&maps.k, a.k, a.Hkv, page, a.num_pages, 1, imin(page, kBN)) ||
        !make_heads_map(&maps.v, a.v, a.Hkv, page, a.num_pages, 1, imin(page, kBN)))
        return LF_ERR_CUDA;
    const long long items = pp.tensor_items(a.T, a.n_seqs, a.Hkv, G);
    // (items counts slots, of which a batch of single tokens fills few)
    if (a.dtype == LF_F16) return launch<__half, true>(maps, a, pp, items, pp.ahead, stream);
    return launch<__nv_bfloat16, true>(maps, a, pp, items, pp.ahead, stream);
}

}  // namespace lf
