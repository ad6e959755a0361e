// Appending new tokens to a paged key/value cache.
//
// Token t of sequence b's n_b new ones goes to position kv_lens[b] - n_b + t.
// A copy, bound by HBM (and by its launch for a few tokens): 8 threads move
// one 128-byte row of k and of v with 16-byte accesses.  4.6 us for 2048
// tokens of 4 heads, as for one.
#include "lf_tc_tiles.cuh"

namespace lf {
namespace {

constexpr int kRowsPerBlock = 32;

__global__ void __launch_bounds__(kRowsPerBlock * 8) append_kernel(const __grid_constant__ PagedArgs a) {
    sm100::pdl_launch_dependents();
    sm100::pdl_wait();
    const int part = threadIdx.x & 7;
    const long long row = (long long)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 3);  // (token, kv head)
    if (blockIdx.x == 0) check_lengths(a.cu, nullptr, a.n_seqs, a.T, a.status, threadIdx.x, blockDim.x);
    const int tok = imin((int)(row / a.Hkv), a.T - 1), h = (int)(row % a.Hkv);
    // a warp holds four rows, of tokens in order: the first one's sequence
    // is the others' too, or they search on from it
    int b = seq_of_token_warp(a.cu, a.n_seqs, __shfl_sync(0xffffffffu, tok, 0));
    while (b + 1 < a.n_seqs && a.cu[b + 1] <= tok) ++b;
    if (row >= (long long)a.T * a.Hkv) return;
    if (tok < a.cu[b] || tok >= a.cu[b + 1]) return;  // behind the last sequence
    const int j = a.kv_lens[b] - (a.cu[b + 1] - tok);
    const int page = page_of(a.table + (size_t)b * a.max_pages, a.max_pages, a.num_pages, a.page_shift, j);
    if (page < 0) {
        if (part == 0) record_status(a.status, b, j < 0 ? LF_ERR_BAD_LENGTHS : LF_ERR_BAD_PAGE);
        return;
    }
    const int slot = j & ((1 << a.page_shift) - 1);
    auto at = [&](const lf_heads& v, int batch, int token) {
        return reinterpret_cast<uint4*>(static_cast<uint16_t*>(v.data) + batch * v.batch_stride + h * v.head_stride +
                                        token * v.token_stride) + part;
    };
    const uint4 k = *at(a.k_new, 0, tok), v = *at(a.v_new, 0, tok);
    *at(a.k, page, slot) = k;
    *at(a.v, page, slot) = v;
}

}  // namespace

lf_status launch_paged_append(const PagedArgs& a, cudaStream_t stream) {
    const long long rows = (long long)a.T * a.Hkv;
    return launch_pdl(append_kernel, dim3((unsigned)((rows + kRowsPerBlock - 1) / kRowsPerBlock)),
                      dim3(kRowsPerBlock * 8), 0, stream, a);
}

}  // namespace lf
