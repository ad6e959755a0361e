// Windowed causal attention with sinks, backward, on the sm_100a tensor cores
// (fp16 / bf16).  P is recomputed from the saved log-sum-exp, so no pass over
// the keys needs a running maximum:
//     P = 2^(S - lse),  dP = dO V^T,  dS = P (dP - delta),  delta = rowsum(dO * out)
//
// dq_kernel     one CTA per 128 query rows (128 / G tokens x G heads), over
//               the blocks of 64 keys it sees:  dQ += dS K.  Writes delta.
// dkv_kernel    128 keys at a time, over the tiles of 64 query rows that hold
//               them in their window, all G heads of the group:
//                   dV += P^T dO,  dK += dS^T Q
//               with S^T = K Q^T and dP^T = V dO^T, so that P^T and dS^T land
//               with keys on the tensor-memory lanes, ready as A operands.
//               Other items of the same launch are the sink keys over a chunk
//               of the queries outside their window: fp32 partials.
// Two kernels compute S and dP twice (7 products instead of 5) but every sum
// has one owner: no atomics, the results repeat bit for bit, and neither dQ
// nor dK, dV ever leaves tensor memory unfinished.
//
// The 8 math warps split a tile's columns in halves (two threads a row), the
// 16-bit P or dS of a half overwriting the first 16 columns of that half's
// scores.  256 tensor-memory columns a CTA, two CTAs per SM, which is what
// bounds both kernels: a dK, dV step is a chain of 2700 cycles, 1650 with the
// other CTA's between, of which the exponentials and the products take about
// 500 each.  (A third of the exponentials on the FMA pipe, 13 instructions a
// pair, and selects in tiles without a mask cost 40 % of a pass.)  16384
// packed tokens, 16 / 4 heads, window 1024, bf16: dQ 153 us, dK and dV 241;
// 16384 tokens, 12 heads, window 256, 32 sinks, fp16: 73 and 99.  P and dS
// are rounded to the storage type, the MMA's operand type; accumulators are
// fp32, rounded once.  dS is about |dout| P: fp16 keeps its bits where the
// loss is scaled so that dout is of order one, as fp16 training does (errors of
// dQ in those of gradients rounded once, window 1024: dout of order 1 1.45,
// 1e-3 3.0, 1e-4 3.6; bf16 has the range).
//
// Rows of other sequences (or of no token) that a tile's loads bring along
// are zeroed in shared memory where they are a product's inner dimension:
// their P is 0, but 0 * NaN is not.
#include <atomic>

#include "lf_tc_tiles.cuh"

namespace lf {
namespace {

using namespace sm100;

constexpr int kD = 64;
constexpr int kStages = 3;
constexpr int kMathWarps = 8;
constexpr int kThreads = (kMathWarps + 2) * 32;  // warp 8: TMA, warp 9: MMA
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kBig = 128 * kD * 2, kSmall = 64 * kD * 2;
constexpr float kLog2e = 1.4426950408889634f;

// Shared memory: two stationary tiles (128 rows), kStages pairs of moving
// tiles (64 rows), per-row constants, barriers.
constexpr uint32_t kOffB = 2 * kBig;                       // moving: stage s, tile 0 / 1
constexpr uint32_t kOffRow = kOffB + kStages * 2 * kSmall; // floats
constexpr uint32_t kRowFloats = kStages * 128;
constexpr int kRing = 4;                                   // items ahead
constexpr uint32_t kPlanBytes = 64;
constexpr uint32_t kOffPlan = kOffRow + kRowFloats * 4;
constexpr uint32_t kOffBar = kOffPlan + kRing * kPlanBytes;
constexpr uint32_t kBars = 2 + 2 * kStages + 8 + 2 * kRing;
constexpr uint32_t kOffMisc = kOffBar + kBars * 8;
constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;      // + alignment slack
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");

// CTAs that run at once.  dK, dV: from kRounds rounds of items of at most
// kShort steps on, that many CTAs take every kResident-th item; else an item
// is a CTA of its own.  Both ways, the backward of 16384 tokens x 12 heads (5
// rounds): window 256 (6 steps) 150 and 159 us, 1024 (18) 295 and 300, 2048
// (34) 491 and 475; 2 rounds of ragged items up to 72 steps 444 and 368.
constexpr int kResident = 2 * 148, kRounds = 3, kShort = 20;

struct Maps {
    CUtensorMap q, k, v, dout;  // stationary or moving boxes, per kernel
};

struct Ctx {
    uint8_t* smem;
    uint64_t *a_full, *a_empty, *b_full, *b_empty, *s_full, *dp_full, *free_, *ready, *done, *drain, *halves, *plan_full, *plan_empty;
    volatile int* abort_flag;
    uint32_t tmem;
};

// Barriers and tensor memory.  `ready_count`: arrivals of a math step.
__device__ __forceinline__ Ctx setup(uint8_t* smem, int warp, int lane) {
    Ctx c;
    c.smem = smem;
    c.a_full = reinterpret_cast<uint64_t*>(smem + kOffBar);
    c.a_empty = c.a_full + 1;
    c.b_full = c.a_empty + 1;
    c.b_empty = c.b_full + kStages;
    c.s_full = c.b_empty + kStages;
    c.dp_full = c.s_full + 1;
    c.free_ = c.dp_full + 1;
    c.ready = c.free_ + 1;  // [2]
    c.done = c.ready + 2;
    c.drain = c.done + 1;
    c.halves = c.drain + 1;
    c.plan_full = c.halves + 1;
    c.plan_empty = c.plan_full + kRing;
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
    c.abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
    if (threadIdx.x == 0) {
        mbar_init(c.a_full, 1);
        mbar_init(c.a_empty, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&c.b_full[s], 1);
            mbar_init(&c.b_empty[s], 1);
        }
        mbar_init(c.s_full, 1);
        mbar_init(c.dp_full, 1);
        mbar_init(c.free_, kMathWarps);
        mbar_init(&c.ready[0], kMathWarps);
        mbar_init(&c.ready[1], kMathWarps);
        mbar_init(c.done, 1);
        mbar_init(c.drain, 1);
        mbar_init(c.halves, kMathWarps);
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&c.plan_full[s], 1);
            mbar_init(&c.plan_empty[s], kMathWarps + 1);
        }
        *c.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMathWarps + 1) {
        tmem_alloc(slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    c.tmem = __shfl_sync(0xffffffffu, *slot, 0);
    return c;
}

__device__ __forceinline__ void finish(const Ctx& c, int warp, int* status) {
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *c.abort_flag) record_status(status, 0, LF_ERR_DEVICE_TIMEOUT);
    if (warp == kMathWarps + 1) {
        tc_fence_after();
        tmem_dealloc(c.tmem, kTmemCols);
    }
}

// Wind-down after an abort: issued copies land, issued MMAs end.
__device__ __forceinline__ void drain_loads(const Ctx& c, int items, int issued) {
    volatile int never = 0;
    if (items > 0) mbar_wait(c.a_full, (items - 1) & 1, &never, 200000000ull);
    for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
        mbar_wait(&c.b_full[j % kStages], (j / kStages) & 1, &never, 200000000ull);
}
__device__ __forceinline__ void drain_mmas(const Ctx& c) {
    volatile int never = 0;
    commit_elect(c.drain);
    mbar_wait(c.drain, 0, &never, 200000000ull);
}

// D = A B^T, both 64 wide and K-major in shared memory (M 128, N 64).
template <typename T>
__device__ __forceinline__ void mma_nt(uint32_t d, uint32_t a_smem, uint32_t b_smem) {
    mma4_ss(d, desc_sw128(a_smem), desc_sw128(b_smem), idesc_f16(MmaFormat<T>::fmt, 128, 64, 0, 0));
}
// D += A B: A (128 x 64, 16-bit) in tensor memory, its halves 32 columns
// apart; B 64 x 64 in shared memory.
template <typename T>
__device__ __forceinline__ void mma_tn(uint32_t d, uint32_t a_tmem, uint32_t b_smem, bool accumulate) {
    mma4_ts(d, d, a_tmem, desc_sw128(b_smem, 0), idesc_f16(MmaFormat<T>::fmt, 128, 64, 0, 1), accumulate, 1);
}

// Zero the rows [from, 64) of a 64-row tile (256 math threads).
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from) {
    const int row = threadIdx.x >> 2;
    if (row >= from) {
        uint4* z = reinterpret_cast<uint4*>(tile + row * 128 + (threadIdx.x & 3) * 32);
        z[0] = z[1] = make_uint4(0u, 0u, 0u, 0u);
    }
}

__device__ __forceinline__ uint8_t* smem_base() {
    extern __shared__ uint8_t raw[];
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
}

// ---------------------------------------------------------------- dQ
// delta comes from out as it was rounded to 16 bits, except where a row may
// see few keys: there dP and delta nearly cancel, and the rounding would be
// much of dS.  Such tiles take their blocks twice, and the first pass sums
// delta = sum P dP in fp32.  They are the tiles of a call whose rows see at
// most kFewKeys keys, sinks among them, and the first of a sequence (up to
// kTwice blocks).  Errors of dQ, in those of gradients rounded once, with
// delta from fp32 and from the rounded out (bf16, emulated): 2 keys 1.4 and
// 2.2, 3 keys 1.4 and 1.9, 6 keys 1.4 and 1.6, 20 keys 1.41 and 1.48, 132 keys
// 1.40 and 1.44.  What is left is dS as a 16-bit operand.
constexpr int kTwice = 3, kFewKeys = 32;

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
dq_kernel(const __grid_constant__ Maps maps, const __grid_constant__ WindowArgs a) {
    uint8_t* smem = smem_base();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int G = a.Hq / a.Hkv, TQ = 128 / G, hk = blockIdx.y;
    if (blockIdx.x == 0 && hk == 0) check_lengths(a.cu, a.lens, a.n_seqs, a.L, a.status, threadIdx.x, blockDim.x);
    // long rows of a causal sequence first
    const TokenTile t = token_tile(a.cu, a.lens, a.n_seqs, a.L, TQ, gridDim.x - 1 - blockIdx.x);
    if (t.t0 >= t.rows) return;
    const int r = (warp & 3) * 32 + lane, half = warp >> 2;  // math warps: row, column half
    const int tok = t.t0 + r / G, head = hk * G + r % G;
    const bool stored = warp < kMathWarps && r < TQ * G && tok < t.rows;
    const bool live = stored && tok < t.n;
    T* dq = view_row<T>(a.dq, t.batch, head, t.start + tok) + half * 32;
    if (t.t0 >= t.n) {  // padding
        if (stored)
#pragma unroll
            for (int c = 0; c < 4; ++c) reinterpret_cast<uint4*>(dq)[c] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const int i0 = t.t0, i1 = imin(t.t0 + TQ, t.n) - 1;
    const KeyBlocks kb = key_blocks(i0, i1, t.n, a.w, a.sinks, 64);
    const bool few = kb.n <= kTwice || a.w + 1 + a.sinks <= kFewKeys;
    const int first = few ? kb.n : 0, steps = first + kb.n;  // steps of the first pass, of both
    auto key0 = [&](int j) { return key_block(kb, j < first ? j : j - first) * 64; };
    const Ctx c = setup(smem, warp, lane);
    const uint32_t tmS = c.tmem, tmP = c.tmem + 128, tmQ = c.tmem + 192;
    float* row_s = reinterpret_cast<float*>(smem + kOffRow);

    if (warp == kMathWarps) {
        // ------------------------------------------------------------ TMA
        if (lane == 0) {
            mbar_arrive_expect_tx(c.a_full, 2 * (uint32_t)(TQ * G) * kD * 2);
            tma_load_4d(smem, &maps.q, c.a_full, 0, hk * G, t.start + t.t0, t.batch);
            tma_load_4d(smem + kBig, &maps.dout, c.a_full, 0, hk * G, t.start + t.t0, t.batch);
        }
        bool ok = true;
        int j = 0;
        for (; j < steps; ++j) {
            const int s = j % kStages;
            ok = warp_wait(&c.b_empty[s], ((j / kStages) & 1) ^ 1, c.abort_flag);
            if (!ok) break;
            if (lane == 0) {
                uint8_t* d = smem + kOffB + s * 2 * kSmall;
                const int row = t.start + key0(j);
                mbar_arrive_expect_tx(&c.b_full[s], 2 * kSmall);
                tma_load_4d(d, &maps.k, &c.b_full[s], 0, hk, row, t.batch);
                tma_load_4d(d + kSmall, &maps.v, &c.b_full[s], 0, hk, row, t.batch);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) drain_loads(c, 1, j);
    } else if (warp == kMathWarps + 1) {
        // ------------------------------------------------------------ MMA
        // S alternates between two buffers; S and dP of block j + 1 are issued
        // as soon as the math warps have read dP of block j, before dQ of j.
        const uint32_t b0 = smem_u32(smem + kOffB);
        bool ok = warp_wait(c.a_full, 0, c.abort_flag);
        auto scores = [&](int j) -> bool {
            const int s = j % kStages;
            if (!warp_wait(&c.b_full[s], (j / kStages) & 1, c.abort_flag)) return false;
            if (j > 0 && !warp_wait(c.free_, (j - 1) & 1, c.abort_flag)) return false;
            tc_fence_after();
            mma_nt<T>(tmS + (j & 1) * 64, smem_u32(smem), b0 + s * 2 * kSmall);
            mma_nt<T>(tmP, smem_u32(smem + kBig), b0 + s * 2 * kSmall + kSmall);
            commit_elect(c.s_full);
            if (j < first) commit_elect(&c.b_empty[s]);
            return true;
        };
        ok = ok && scores(0);
        for (int j = 0; j < steps && ok; ++j) {
            if (j + 1 < steps) ok = scores(j + 1);
            if (j < first) continue;
            ok = ok && warp_wait(&c.ready[j & 1], ((j >> 1) - ((first + 1 - (j & 1)) >> 1)) & 1, c.abort_flag);
            if (!ok) break;
            tc_fence_after();
            mma_tn<T>(tmQ, tmS + (j & 1) * 64, b0 + (j % kStages) * 2 * kSmall, j > first);
            commit_elect(&c.b_empty[j % kStages]);
            if (j == steps - 1) commit_elect(c.done);
        }
        if (!ok) drain_mmas(c);
    } else {
        // ------------------------------------------------------------ math
        // delta: two threads a row, half of the sum each
        float part = 0.0f, nlse = 0.0f;
        const size_t at = ((size_t)t.batch * a.Hq + head) * a.L + t.start + tok;
        if (live) nlse = -a.lse[at] * kLog2e;
        if (live && first == 0) {
            const size_t off = (((size_t)t.batch * a.L + t.start + tok) * a.Hq + head) * kD + half * 32;
            const uint4* po = reinterpret_cast<const uint4*>(static_cast<const T*>(a.out) + off);
            const uint4* pd = reinterpret_cast<const uint4*>(static_cast<const T*>(a.dout) + off);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint4 x = po[u], y = pd[u];
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = Pair<T>::unpack(xs[e]), g = Pair<T>::unpack(ys[e]);
                    part = fmaf(f.x, g.x, fmaf(f.y, g.y, part));
                }
            }
        }
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const float sc = a.scale * kLog2e;
        const float2 sc2 = make_float2(sc, sc), nl2 = make_float2(nlse, nlse);
        // blocks that every row of this warp sees whole begin in [full_lo, full_hi]
        const bool warp_live = __all_sync(0xffffffffu, live);
        const int full_lo = i1 - a.w, full_hi = imin(i0 + 1, t.n) - 64;
        bool ok = true;
        for (int j = 0; j < first; ++j) {
            const int c0 = key0(j) + 32 * half;
            ok = warp_wait(c.s_full, j & 1, c.abort_flag);
            if (!ok) break;
            tc_fence_after();
            float x[32], y[32];
            tmem_ld32f(tmS + lane_off + (j & 1) * 64 + half * 32, x);
            tmem_ld32f(tmP + lane_off + half * 32, y);
            tmem_ld_wait();
            regs_ready<32>(x);
            regs_ready<32>(y);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.free_);
            const uint32_t bits = live ? visible_bits32(tok, c0, t.n, a.w, a.sinks) : 0u;
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if ((bits >> e) & 1) part = fmaf(ex2(fmaf(x[e], sc, nlse)), y[e], part);
        }
        row_s[half * 128 + r] = part;
        __syncwarp();
        if (lane == 0) mbar_arrive(c.halves);
        ok = ok && warp_wait(c.halves, 0, c.abort_flag);
        const float ndelta = ok ? -(row_s[r] + row_s[128 + r]) : 0.0f;
        if (live && half == 0) a.delta[at] = -ndelta;
        const float2 nd2 = make_float2(ndelta, ndelta);
        for (int j = first; j < steps && ok; ++j) {
            const int c0 = key0(j);
            const uint32_t tS = tmS + lane_off + (j & 1) * 64 + half * 32;
            const bool full = warp_live && c0 <= full_hi && c0 >= full_lo;
            ok = warp_wait(c.s_full, j & 1, c.abort_flag);
            if (!ok) break;
            tc_fence_after();
            float x[32], y[32];
            tmem_ld32f(tS, x);
            tmem_ld32f(tmP + lane_off + half * 32, y);
            tmem_ld_wait();
            regs_ready<32>(x);
            regs_ready<32>(y);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.free_);
            uint32_t pk[16];
            if (full) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 v = ffma2(make_float2(x[2 * e], x[2 * e + 1]), sc2, nl2);
                    const float2 d = fmul2(make_float2(ex2(v.x), ex2(v.y)), fadd2(make_float2(y[2 * e], y[2 * e + 1]), nd2));
                    pk[e] = Pair<T>::pack(d.x, d.y);
                }
            } else {
                const uint32_t bits = live ? visible_bits32(tok, c0 + 32 * half, t.n, a.w, a.sinks) : 0u;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 v = ffma2(make_float2(x[2 * e], x[2 * e + 1]), sc2, nl2);
                    const float2 d = fmul2(make_float2(ex2(v.x), ex2(v.y)), fadd2(make_float2(y[2 * e], y[2 * e + 1]), nd2));
                    pk[e] = Pair<T>::pack((bits >> (2 * e)) & 1 ? d.x : 0.0f, (bits >> (2 * e + 1)) & 1 ? d.y : 0.0f);
                }
            }
            tmem_st16(tS, pk);
            if (c0 + 64 > t.n) {  // keys past the sequence
                zero_rows(smem + kOffB + (j % kStages) * 2 * kSmall, t.n - c0);
                fence_proxy_async_smem();
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.ready[j & 1]);
        }
        if (ok && warp_wait(c.done, 0, c.abort_flag)) {
            tc_fence_after();
            float o[32];
            tmem_ld32f(tmQ + lane_off + half * 32, o);
            tmem_ld_wait();
            regs_ready<32>(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= a.scale;
            if (live) store_row32(dq, o);
            else if (stored)
#pragma unroll
                for (int u = 0; u < 4; ++u) reinterpret_cast<uint4*>(dq)[u] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    finish(c, warp, a.status);
}

// ---------------------------------------------------------------- dK, dV
// P is an operand of dV as P 2^kLift: of rows that see more than 2^14 keys, P
// would fall among fp16's subnormal numbers (1 / 48000 is off by 2^-10 there).
// Lifted, it keeps its bits down to 2^-24, and stays finite up to 2^6 (scores
// that large lose bits in fp32 first).  The lift is part of the exponent's
// offset and of the factor of dP - delta, so it costs no instruction but the
// last products of dV.
template <typename T>
constexpr int kLift = MmaFormat<T>::fmt == 0 ? 10 : 0;

// What the roles need to know of an item: 128 keys and the query tokens
// [q0, q1) that its dK and dV sum over.  nq: steps; 0: rows of zeros
// (padding, or a chunk inside every window), < 0: no more items.
struct KeyItem {
    int nq, c0, q0, q1;       // first key
    int n_keys, n_sink;       // keys from here on get nothing; keys up to here have partials
    int hk, b, chunk;         // key/value head, sequence; its chunk of queries
    int batch, start, n, rows;
    int sink;                 // a chunk of queries outside the window of its sink keys
    int use;                  // items with steps before this one
};
static_assert(sizeof(KeyItem) <= kPlanBytes, "plan slot");

// false: the item has no work at all.
__device__ __forceinline__ bool key_item(const WindowArgs& a, int item, int sink_slots, int sink_items, int per_head, int TQ,
                                         KeyItem& p) {
    // the sink chunks come first: they are the longest items
    const int n_first = sink_items * a.Hkv;
    p.sink = item < n_first;
    int slot, at = p.sink ? item : item - n_first;
    const int per = p.sink ? sink_items : per_head;
    p.hk = at / per;
    at -= p.hk * per;
    slot = p.sink ? at % sink_slots : at;
    const TokenTile t = token_tile(a.cu, a.lens, a.n_seqs, a.L, p.sink ? a.chunk : 128, slot);
    if (t.t0 >= (p.sink ? t.n : t.rows)) return false;
    p.n_sink = a.sink().any(t.n) ? imin(a.sinks, t.n) : 0;
    p.b = t.b;
    p.chunk = 0;
    if (p.sink) {
        p.chunk = t.t0 / a.chunk;
        if (p.n_sink == 0 || p.chunk < a.sink().first_chunk()) return false;
        p.c0 = at / sink_slots * 128;
        if (p.c0 >= p.n_sink) return false;  // (more sinks than the sequence has)
        p.q0 = imax(t.t0, p.c0 + a.w + 1);
        p.q1 = imin(t.t0 + a.chunk, t.n);
        p.n_keys = p.n_sink;
    } else {
        p.c0 = p.q0 = t.t0;
        p.q1 = (int)min((long long)t.n, (long long)p.c0 + 128 + a.w);
        p.n_keys = t.n;
    }
    p.nq = p.q1 > p.q0 ? (p.q1 - p.q0 + TQ - 1) / TQ : 0;
    p.batch = t.batch;
    p.start = t.start;
    p.n = t.n;
    p.rows = t.rows;
    return true;
}

// kMany: CTAs take several items each; the next one's plan, loads and first
// products run under the end of the last.  Else a CTA has one, whose bounds
// are uniform values: a step is 4 % shorter than with bounds that come through
// shared memory.
template <typename T, bool kMany>
__global__ void __launch_bounds__(kThreads, 2)
dkv_kernel(const __grid_constant__ Maps maps, const __grid_constant__ WindowArgs a, int sink_slots, int sink_items,
           int per_head, int n_items) {
    uint8_t* smem = smem_base();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int G = a.Hq / a.Hkv, TQ = 64 / G;
    constexpr float kDrop = 1.0f / (1 << kLift<T>);
    [[maybe_unused]] KeyItem own;
    if constexpr (!kMany) {
        if (!key_item(a, blockIdx.x, sink_slots, sink_items, per_head, TQ, own)) return;
        own.use = 0;
    }
    if (TQ * G < 64 && warp < kMathWarps) {  // rows no load ever writes
        for (int s = 0; s < 2 * kStages; ++s) zero_rows(smem + kOffB + s * kSmall, TQ * G);
        fence_proxy_async_smem();
    }
    const Ctx c = setup(smem, warp, lane);
    const uint32_t tmS = c.tmem, tmP = c.tmem + 64, tmV = c.tmem + 128, tmK = c.tmem + 192;
    float* row_s = reinterpret_cast<float*>(smem + kOffRow);  // [stage][kLift - lse log2e, -delta kDrop][64]
    auto plan_slot = [&](int k) { return reinterpret_cast<KeyItem*>(smem + kOffPlan + (k % kRing) * kPlanBytes); };
    // The items, in order; the slot of item k - 1 is handed back when the
    // role asks for item k.  NULL at the end and after an abort.
    auto next_item = [&](int k, bool& ok) -> const KeyItem* {
        if constexpr (!kMany) return k == 0 ? &own : nullptr;
        if (k > 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.plan_empty[(k - 1) % kRing]);
        }
        ok = warp_wait(&c.plan_full[k % kRing], (k / kRing) & 1, c.abort_flag);
        return ok && plan_slot(k)->nq >= 0 ? plan_slot(k) : nullptr;
    };

    if (warp == kMathWarps) {
        // ------------------------------------------------------------ TMA
        // Plans an item and publishes it while the last one's loaded steps
        // are worked on.
        bool ok = true;
        int g = 0, it = 0, k = 0;  // steps, items with steps, items so far
        for (int item = blockIdx.x; ok; item += gridDim.x) {
            KeyItem p;
            if constexpr (kMany) {
                p.nq = -1;
                if (item < n_items && !key_item(a, item, sink_slots, sink_items, per_head, TQ, p)) continue;
                ok = warp_wait(&c.plan_empty[k % kRing], ((k / kRing) & 1) ^ 1, c.abort_flag);
                if (!ok) break;
                p.use = it;
                if (lane == 0) {
                    *plan_slot(k) = p;
                    mbar_arrive(&c.plan_full[k % kRing]);
                }
                ++k;
            } else {
                p = own;
                if (item != (int)blockIdx.x) break;
            }
            if (p.nq < 0) break;
            if (p.nq == 0) continue;
            ok = warp_wait(c.a_empty, (it & 1) ^ 1, c.abort_flag);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(c.a_full, 2 * kBig);
                tma_load_4d(smem, &maps.k, c.a_full, 0, p.hk, p.start + p.c0, p.batch);
                tma_load_4d(smem + kBig, &maps.v, c.a_full, 0, p.hk, p.start + p.c0, p.batch);
            }
            ++it;
            for (int j = 0; j < p.nq; ++j, ++g) {
                const int s = g % kStages, qt = p.q0 + j * TQ;
                // this lane's two rows
                float nl[2], nd[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int row = lane + 32 * u, tok = qt + row / G;
                    const bool live = row < TQ * G && tok < p.q1;
                    const size_t at = ((size_t)p.batch * a.Hq + p.hk * G + row % G) * a.L + p.start + tok;
                    nl[u] = live ? fmaf(-a.lse[at], kLog2e, (float)kLift<T>) : 0.0f;
                    nd[u] = live ? -a.delta[at] * kDrop : 0.0f;
                }
                ok = warp_wait(&c.b_empty[s], ((g / kStages) & 1) ^ 1, c.abort_flag);
                if (!ok) break;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    row_s[s * 128 + lane + 32 * u] = nl[u];
                    row_s[s * 128 + 64 + lane + 32 * u] = nd[u];
                }
                __syncwarp();
                if (lane == 0) {
                    uint8_t* d = smem + kOffB + s * 2 * kSmall;
                    mbar_arrive_expect_tx(&c.b_full[s], 2 * (uint32_t)(TQ * G) * kD * 2);
                    tma_load_4d(d, &maps.q, &c.b_full[s], 0, p.hk * G, p.start + qt, p.batch);
                    tma_load_4d(d + kSmall, &maps.dout, &c.b_full[s], 0, p.hk * G, p.start + qt, p.batch);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) drain_loads(c, it, g);
    } else if (warp == kMathWarps + 1) {
        // ------------------------------------------------------------ MMA
        // In issue order S_0, dP_0, then per tile dV_j, S_(j+1) once P is
        // there and dK_j, dP_(j+1) once dS is: S_(j+1) may overwrite P_j, and
        // dP_(j+1) dS_j, without a wait, and each pair runs under the other
        // half of the math warps' step.  S_0 and dP_0 of the next item run
        // under the last one's epilogue; its first dV and dK overwrite the
        // sums, after the P and dS of warps that have read them.
        constexpr uint32_t id_nt = idesc_f16(MmaFormat<T>::fmt, 128, 64, 0, 0), id_tn = idesc_f16(MmaFormat<T>::fmt, 128, 64, 0, 1);
        const uint64_t dk = desc_sw128(smem_u32(smem)), dv = desc_sw128(smem_u32(smem + kBig)),
                       q_nt = desc_sw128(smem_u32(smem + kOffB)), q_tn = desc_sw128(smem_u32(smem + kOffB), 0);
        constexpr uint32_t kHop = 2 * kSmall >> 4, kDo = kSmall >> 4;  // to the next stage, to its dO
        bool ok = true;
        int g = 0, it = 0, s = 0, phase = 0;  // steps, items with steps; stage and its use
        for (int k = 0; ok; ++k) {
            const KeyItem* p = next_item(k, ok);
            if (!p) break;
            int left = p->nq;
            if (left == 0) continue;
            ok = warp_wait(c.a_full, it & 1, c.abort_flag) && warp_wait(&c.b_full[s], phase, c.abort_flag);
            if (!ok) break;
            tc_fence_after();
            mma4_ss(tmS, dk, q_nt + s * kHop, id_nt);
            commit_elect(c.s_full);
            mma4_ss(tmP, dv, q_nt + s * kHop + kDo, id_nt);
            commit_elect(c.dp_full);
            if (left == 1) commit_elect(c.a_empty);
            uint32_t accumulate = 0;
            for (; left > 0; --left, ++g) {
                const int s0 = s;
                const uint64_t q = q_tn + s0 * kHop;
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1;
                }
                const uint64_t next = q_nt + s * kHop;
                const bool more = left > 1;
                ok = (!more || warp_wait(&c.b_full[s], phase, c.abort_flag)) && warp_wait(&c.ready[0], g & 1, c.abort_flag);
                if (!ok) break;
                tc_fence_after();
                mma4_ts(tmV, tmV, tmS, q + kDo, id_tn, accumulate, 1);
                if (more) {
                    mma4_ss(tmS, dk, next, id_nt);
                    commit_elect(c.s_full);
                }
                ok = warp_wait(&c.ready[1], g & 1, c.abort_flag);
                if (!ok) break;
                tc_fence_after();
                mma4_ts(tmK, tmK, tmP, q, id_tn, accumulate, 1);
                if (more) {
                    mma4_ss(tmP, dv, next + kDo, id_nt);
                    commit_elect(c.dp_full);
                }
                commit_elect(&c.b_empty[s0]);
                if (left == 2) commit_elect(c.a_empty);
                if (!more) commit_elect(c.done);
                accumulate = 1;
            }
            ++it;
        }
        if (!ok) drain_mmas(c);
    } else {
        // ------------------------------------------------------------ math
        const int r = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmS + lane_off + half * 32, tP = tmP + lane_off + half * 32;
        const float sc = a.scale * kLog2e;
        const float2 sc2 = make_float2(sc, sc);
        bool ok = true;
        int g = 0;
        for (int k = 0; ok; ++k) {
            const KeyItem* p = next_item(k, ok);
            if (!p) break;
            const int key = p->c0 + r;
            // Where this thread's half rows of dK and dV go: the fp32 partials
            // of a sink key, or the outputs (worked out when they are needed).
            struct Target {
                float* part;
                T *dk, *dv;
            };
            auto target = [&]() -> Target {
                Target o = {nullptr, nullptr, nullptr};
                if (key < p->n_sink) {
                    const int start = a.cu ? p->start : p->b * a.L;
                    const long long row = p->sink ? a.sink().chunk_row(p->b, start, p->chunk) : a.sink().own(p->b, start);
                    o.part = a.part + ((size_t)p->hk * a.sink().rows() + row + key) * 2 * kD + half * 32;
                } else if (!p->sink && key < p->rows) {
                    o.dk = view_row<T>(a.dk, p->batch, p->hk, p->start + key) + half * 32;
                    o.dv = view_row<T>(a.dv, p->batch, p->hk, p->start + key) + half * 32;
                }
                return o;
            };
            if (p->nq == 0) {
                const Target o = target();
                if (o.part) {
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        reinterpret_cast<float4*>(o.part)[u] = reinterpret_cast<float4*>(o.part + kD)[u] =
                            make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (o.dk) {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        reinterpret_cast<uint4*>(o.dk)[u] = reinterpret_cast<uint4*>(o.dv)[u] = make_uint4(0u, 0u, 0u, 0u);
                }
                continue;
            }
            // (kMany: what a step needs of the item stays in shared memory,
            // registers are short)
            for (int qt = p->q0; qt < p->q1; qt += TQ, ++g) {
                const int s = g % kStages;
                // columns (query rows) that see this thread's key: tokens from
                // the key on to the window's end, or past it for a sink
                const int past = iclamp(key + a.w + 1 - qt, 0, 64) * G, end = imin(p->q1 - qt, TQ) * G;
                const int lo = p->sink ? past : iclamp(key - qt, 0, 64) * G, hi = p->sink ? end : imin(past, end);
                const uint32_t bits = key < p->n_keys ? low_bits32(hi - 32 * half) & ~low_bits32(lo - 32 * half) : 0u;
                const bool full = __all_sync(0xffffffffu, bits == ~0u);
                const float4* nl4 = reinterpret_cast<const float4*>(row_s + s * 128 + half * 32);
                const float4* nd4 = nl4 + 16;
                ok = warp_wait(c.s_full, g & 1, c.abort_flag) && warp_wait(&c.b_full[s], (g / kStages) & 1, c.abort_flag);
                if (!ok) break;
                tc_fence_after();
                // P 2^kLift, kept in fp32 for dS
                float x[32];
                uint32_t pk[16];
                tmem_ld32f(tS, x);
                tmem_ld_wait();
                regs_ready<32>(x);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float4 nl = nl4[u];
                    const float2 v0 = ffma2(make_float2(x[4 * u], x[4 * u + 1]), sc2, make_float2(nl.x, nl.y));
                    const float2 v1 = ffma2(make_float2(x[4 * u + 2], x[4 * u + 3]), sc2, make_float2(nl.z, nl.w));
                    x[4 * u] = ex2(v0.x);
                    x[4 * u + 1] = ex2(v0.y);
                    x[4 * u + 2] = ex2(v1.x);
                    x[4 * u + 3] = ex2(v1.y);
                }
                if (!full) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = (bits >> e) & 1 ? x[e] : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = Pair<T>::pack(x[2 * e], x[2 * e + 1]);
                tmem_st16(tS, pk);
                if (qt + TQ > p->n) {  // query rows past the sequence
                    // (dP reads dO: only what is of no use to it changes, but not under it)
                    ok = warp_wait(c.dp_full, g & 1, c.abort_flag);
                    if (!ok) break;
                    uint8_t* d = smem + kOffB + s * 2 * kSmall;
                    zero_rows(d, (p->n - qt) * G);
                    zero_rows(d + kSmall, (p->n - qt) * G);
                    fence_proxy_async_smem();
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.ready[0]);
                // dS
                ok = warp_wait(c.dp_full, g & 1, c.abort_flag);
                if (!ok) break;
                tc_fence_after();
                float y[32];
                tmem_ld32f(tP, y);
                tmem_ld_wait();
                regs_ready<32>(y);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float4 nd = nd4[u];
                    const float2 drop = make_float2(kDrop, kDrop);
                    const float2 d0 = fmul2(make_float2(x[4 * u], x[4 * u + 1]), ffma2(make_float2(y[4 * u], y[4 * u + 1]), drop, make_float2(nd.x, nd.y)));
                    const float2 d1 = fmul2(make_float2(x[4 * u + 2], x[4 * u + 3]), ffma2(make_float2(y[4 * u + 2], y[4 * u + 3]), drop, make_float2(nd.z, nd.w)));
                    y[4 * u] = d0.x;
                    y[4 * u + 1] = d0.y;
                    y[4 * u + 2] = d1.x;
                    y[4 * u + 3] = d1.y;
                }
                if (!full) {  // (0 times what a dead row's dP holds)
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = (bits >> e) & 1 ? y[e] : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = Pair<T>::pack(y[2 * e], y[2 * e + 1]);
                tmem_st16(tP, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.ready[1]);
            }
            if (ok) ok = warp_wait(c.done, p->use & 1, c.abort_flag);
            if (ok) {
                tc_fence_after();
                const Target to = target();
#pragma unroll
                for (int w = 0; w < 2; ++w) {  // dK, dV
                    float o[32];
                    tmem_ld32f((w ? tmV : tmK) + lane_off + half * 32, o);
                    tmem_ld_wait();
                    regs_ready<32>(o);
                    if (w == 0 || kLift<T> > 0) {
                        const float f = w == 0 ? a.scale : kDrop;
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                    }
                    if (to.part) {
                        float4* d = reinterpret_cast<float4*>(to.part + w * kD);
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            d[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
                    } else if (to.dk) {
                        T* d = w ? to.dv : to.dk;
                        if (key < p->n_keys) store_row32(d, o);
                        else
#pragma unroll
                            for (int u = 0; u < 4; ++u) reinterpret_cast<uint4*>(d)[u] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    __syncwarp();
                }
            }
        }
    }
    finish(c, warp, a.status);
}

template <typename K>
lf_status opt_in(K kernel, std::atomic<bool>* done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return LF_ERR_CUDA;
    if (!done[dev].load()) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
            return LF_ERR_CUDA;
        done[dev].store(true);
    }
    return LF_OK;
}

template <typename T>
lf_status backward_t(const WindowArgs& a, cudaStream_t stream) {
    static std::atomic<bool> attr[3][64];
    lf_status st = opt_in(dq_kernel<T>, attr[0]);
    if (st == LF_OK) st = opt_in(dkv_kernel<T, false>, attr[1]);
    if (st == LF_OK) st = opt_in(dkv_kernel<T, true>, attr[2]);
    if (st != LF_OK) return st;
    const int G = a.heads_group(), B = a.packed() ? 1 : a.n_seqs;
    const lf_heads dout = {const_cast<void*>(a.dout), (long long)a.L * a.Hq * kD, kD, (long long)a.Hq * kD};
    Maps mq, mk;
    if (!make_heads_map(&mq.q, a.q, a.Hq, a.L, B, G, 128 / G) ||
        !make_heads_map(&mq.dout, dout, a.Hq, a.L, B, G, 128 / G) ||
        !make_heads_map(&mq.k, a.k, a.Hkv, a.L, B, 1, 64) || !make_heads_map(&mq.v, a.v, a.Hkv, a.L, B, 1, 64) ||
        !make_heads_map(&mk.q, a.q, a.Hq, a.L, B, G, 64 / G) ||
        !make_heads_map(&mk.dout, dout, a.Hq, a.L, B, G, 64 / G) ||
        !make_heads_map(&mk.k, a.k, a.Hkv, a.L, B, 1, 128) || !make_heads_map(&mk.v, a.v, a.Hkv, a.L, B, 1, 128))
        return LF_ERR_CUDA;
    const int slots = a.sinks > 0 ? token_slots(a.packed(), a.n_seqs, a.L, a.chunk) : 0;
    const long long sink_items = (long long)slots * ((a.sinks + 127) / 128);
    const int per_head = token_slots(a.packed(), a.n_seqs, a.L, 128);
    if (sink_items + per_head > kMostItems / a.Hkv) return LF_ERR_TOO_LARGE;
    const long long items = (sink_items + per_head) * a.Hkv;
    st = launch_pdl(dq_kernel<T>, dim3(token_slots(a.packed(), a.n_seqs, a.L, 128 / G), a.Hkv), dim3(kThreads),
                    kSmemBytes, stream, mq, a);
    if (st != LF_OK) return st;
    const bool many = items >= kRounds * kResident && (128LL + a.w) * G <= kShort * 64;
    st = launch_pdl(many ? dkv_kernel<T, true> : dkv_kernel<T, false>, dim3((unsigned)(many ? kResident : items)),
                    dim3(kThreads), kSmemBytes, stream, mk, a, slots, (int)sink_items, per_head, (int)items);
    if (st == LF_OK && a.sinks > 0) st = launch_sink_reduce(a, stream);
    return st;
}

}  // namespace

lf_status launch_window_backward_tc(const WindowArgs& a, cudaStream_t stream) {
    return a.dtype == LF_F16 ? backward_t<__half>(a, stream) : backward_t<__nv_bfloat16>(a, stream);
}

}  // namespace lf
