// attn_api.cu -- the attention entry points of gdn.h: host-side validation, then launches.
#include <cuda_runtime.h>

#include <initializer_list>

#include "api_checks.cuh"
#include "attn_common.cuh"

using gdn::aligned16;
using gdn::AppendArgs;
using gdn::AttnArgs;
using gdn::cuda_status;
using gdn::dtype_ok;
using gdn::esize;
using gdn::head_dim_ok;
using gdn::overlap;
using gdn::Range;

namespace {

int page_shift_of(int32_t page_size) {
    for (int s = 4; s <= 7; ++s)
        if (page_size == (1 << s)) return s;
    return -1;
}

// Heads, head dim and dtype, in the library's order: SHAPE for sizes that are inconsistent,
// UNSUPPORTED for those no kernel takes.
gdn_status check_heads(gdn_dtype io, int32_t HQ, int32_t HKV, int32_t D) {
    if (HQ <= 0 || HKV <= 0 || D <= 0 || HQ % HKV != 0) return GDN_ERR_SHAPE;
    if (!dtype_ok(io) || !head_dim_ok(D)) return GDN_ERR_UNSUPPORTED;
    if (HQ > 1024 || HKV > 1024) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// Positions and tokens are 32-bit in the kernels, which look up to two steps of 128 past the last one.
constexpr int64_t kMaxPositions = (int64_t)INT32_MAX - 255;

// The cache: row numbers (page * page_size + offset) stay within 32 bits, positions below the limit.
gdn_status check_pages(int32_t n_pages, int32_t page_size, int32_t max_pages) {
    if (n_pages < 0 || page_size <= 0 || max_pages < 0) return GDN_ERR_SHAPE;
    if (page_shift_of(page_size) < 0) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)n_pages * page_size > INT32_MAX || (int64_t)max_pages * page_size > kMaxPositions)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

bool all_aligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (p && !aligned16(p)) return false;
    return true;
}

bool any_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (Range o : outs) {
        for (Range i : ins)
            if (overlap(o, i)) return true;
    }
    for (const Range* a = outs.begin(); a != outs.end(); ++a)
        for (const Range* b = a + 1; b != outs.end(); ++b)
            if (overlap(*a, *b)) return true;
    return false;
}

// What the three attention calls have in common once their sizes are checked.
gdn_status check_attn(const AttnArgs& a, gdn_dtype io, size_t need, void* workspace, size_t workspace_bytes) {
    if (a.kv.table && a.kv.n_pages == 0) return GDN_ERR_SHAPE;
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!a.q || !a.kv.k || !a.kv.v || !a.o) return GDN_ERR_NULL;
    if (!all_aligned({a.q, a.kv.k, a.kv.v, a.kv.table, a.kv.kv_lens, a.cu, a.z, a.o, workspace})) return GDN_ERR_ALIGN;
    const size_t row = (size_t)a.D * esize(io);
    const size_t qb = (size_t)a.n_tokens * a.HQ * row;
    const size_t kb = (a.kv.table ? (size_t)a.kv.n_pages << a.kv.page_shift : (size_t)a.n_tokens) * a.HKV * row;
    const Range table{a.kv.table, a.kv.table ? (size_t)a.n_seqs * a.kv.max_pages * 4 : 0};
    const Range lens{a.kv.kv_lens, a.kv.kv_lens ? (size_t)a.n_seqs * 4 : 0};
    const Range cu{a.cu, a.cu ? (size_t)(a.n_seqs + 1) * 4 : 0};
    if (any_overlap({{a.o, qb}, {workspace, workspace_bytes}},
                    {{a.q, qb}, {a.kv.k, kb}, {a.kv.v, kb}, {a.z, a.z ? qb : 0}, table, lens, cu}))
        return GDN_ERR_ALIAS;
    return GDN_OK;
}

size_t prefill_bytes(int64_t n_tokens, int32_t n_seqs, int32_t HQ, int32_t HKV, int32_t D, gdn_dtype io) {
    if (n_tokens < 0 || n_tokens > kMaxPositions || n_seqs < 0 || check_heads(io, HQ, HKV, D) != GDN_OK) return 0;
    // the kernels count tiles (of one token or more, per key-value head) in 32 bits
    if ((n_tokens + n_seqs) * (int64_t)HQ > INT32_MAX) return 0;
    if (io == GDN_BF16 && gdn::attn_tc_supported(HQ, HKV)) return gdn::attn_tc_bytes(n_tokens, n_seqs, HQ, HKV, D);
    return gdn::attn_cudacore_bytes(n_tokens, n_seqs, HQ, HKV, D);
}

// A prompt call whose sizes are checked.
gdn_status run_prefill(const AttnArgs& a, gdn_dtype io, void* workspace, size_t workspace_bytes, void* stream) {
    const size_t need = prefill_bytes(a.n_tokens, a.n_seqs, a.HQ, a.HKV, a.D, io);
    if (need == 0) return GDN_ERR_UNSUPPORTED;
    const gdn_status st = check_attn(a, io, need, workspace, workspace_bytes);
    if (st != GDN_OK) return st;
    if (a.bf16 && gdn::attn_tc_supported(a.HQ, a.HKV)) return cuda_status(gdn::launch_attn_tc(a, (cudaStream_t)stream));
    return cuda_status(gdn::launch_attn_cudacore(a, (cudaStream_t)stream));
}

size_t decode_bytes(int32_t B, int32_t HQ, int32_t HKV, int32_t D, gdn_dtype io) {
    if (B < 0 || check_heads(io, HQ, HKV, D) != GDN_OK) return 0;
    return gdn::attn_decode_bytes(D);
}

}  // namespace

extern "C" {

gdn_status gdn_attn_append(const void* q, const void* k, const void* v, gdn_dtype io_dtype, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const float* inv_freq, int32_t rotary_dim,
                           int32_t interleaved, const int32_t* cu_seqlens, const int32_t* kv_lens,
                           const int32_t* block_table, int64_t n_tokens, int32_t n_seqs, int32_t HQ, int32_t HKV,
                           int32_t D, int32_t n_pages, int32_t page_size, int32_t max_pages, void* q_out,
                           void* k_cache, void* v_cache, void* stream) {
    if (n_tokens < 0 || n_tokens > INT32_MAX || n_seqs < 0) return GDN_ERR_SHAPE;
    if (!cu_seqlens && n_tokens != n_seqs) return GDN_ERR_SHAPE;
    gdn_status st = check_heads(io_dtype, HQ, HKV, D);
    if (st != GDN_OK) return st;
    st = check_pages(n_pages, page_size, max_pages);
    if (st != GDN_OK) return st;
    if (rotary_dim < 0 || rotary_dim > D) return GDN_ERR_SHAPE;
    if (rotary_dim % 16 != 0) return GDN_ERR_UNSUPPORTED;
    if ((q && q_stride < (int64_t)HQ * D) || k_stride < (int64_t)HKV * D || v_stride < (int64_t)HKV * D)
        return GDN_ERR_SHAPE;
    if (n_tokens == 0 || n_seqs == 0) return GDN_OK;
    if (!k || !v || !kv_lens || !block_table || !k_cache || !v_cache || (q != nullptr) != (q_out != nullptr) ||
        (rotary_dim > 0 && !inv_freq))
        return GDN_ERR_NULL;
    const size_t es = esize(io_dtype);
    if (!all_aligned({q, k, v, inv_freq, cu_seqlens, kv_lens, block_table, q_out, k_cache, v_cache}))
        return GDN_ERR_ALIGN;
    if ((q && q_stride * es % 16) || k_stride * es % 16 || v_stride * es % 16) return GDN_ERR_ALIGN;
    const size_t n1 = (size_t)n_tokens - 1;
    const Range rq{q, (n1 * q_stride + (size_t)HQ * D) * es}, rk{k, (n1 * k_stride + (size_t)HKV * D) * es};
    const Range rv{v, (n1 * v_stride + (size_t)HKV * D) * es};
    const Range rqo{q_out, (size_t)n_tokens * HQ * D * es};
    const size_t cb = (size_t)n_pages * page_size * HKV * D * es;
    const Range rkc{k_cache, cb}, rvc{v_cache, cb};
    const Range rf{inv_freq, (size_t)rotary_dim / 2 * 4}, rl{kv_lens, (size_t)n_seqs * 4};
    const Range rt{block_table, (size_t)n_seqs * max_pages * 4};
    const Range rc{cu_seqlens, cu_seqlens ? (size_t)(n_seqs + 1) * 4 : 0};
    if (any_overlap({rqo, rkc, rvc}, {rk, rv, rf, rl, rt, rc})) return GDN_ERR_ALIAS;
    const bool in_place = q && q == q_out && q_stride == (int64_t)HQ * D;
    if (overlap(rq, rkc) || overlap(rq, rvc) || (!in_place && overlap(rq, rqo))) return GDN_ERR_ALIAS;
    const AppendArgs a{q, k, v, q_stride, k_stride, v_stride, inv_freq, rotary_dim, interleaved != 0, cu_seqlens,
                       n_tokens, n_seqs, HQ, HKV, D, q_out, k_cache, v_cache, block_table, kv_lens, n_pages,
                       page_shift_of(page_size), max_pages, io_dtype == GDN_BF16};
    return cuda_status(gdn::launch_attn_append(a, (cudaStream_t)stream));
}

size_t gdn_attn_prefill_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int32_t HQ, int32_t HKV, int32_t D,
                                        gdn_dtype io_dtype) {
    return prefill_bytes(n_tokens, n_seqs, HQ, HKV, D, io_dtype);
}

gdn_status gdn_attn_prefill(const void* q, const void* k, const void* v, gdn_dtype io_dtype,
                            const int32_t* cu_seqlens, int32_t B, int64_t T, int32_t n_seqs, int32_t HQ, int32_t HKV,
                            int32_t D, float scale, const void* z, void* o, void* workspace, size_t workspace_bytes,
                            void* stream) {
    if (B < 0 || T < 0 || T > INT32_MAX || n_seqs < 0 || B * T > INT32_MAX) return GDN_ERR_SHAPE;
    if (cu_seqlens ? B != 1 : n_seqs != B) return GDN_ERR_SHAPE;
    gdn_status st = check_heads(io_dtype, HQ, HKV, D);
    if (st != GDN_OK) return st;
    if (!(scale - scale == 0.f)) return GDN_ERR_SHAPE;
    const int64_t n_tokens = (int64_t)B * T;
    if (n_tokens == 0 || n_seqs == 0) return GDN_OK;
    const AttnArgs a{q, {k, v, nullptr, nullptr, 0, 0, 0}, cu_seqlens, T, n_tokens, n_seqs, HQ, HKV, D, scale, z, o,
                     io_dtype == GDN_BF16, workspace};
    return run_prefill(a, io_dtype, workspace, workspace_bytes, stream);
}

gdn_status gdn_attn_prefill_paged(const void* q, gdn_dtype io_dtype, const void* k_cache, const void* v_cache,
                                  const int32_t* block_table, const int32_t* kv_lens, const int32_t* cu_seqlens,
                                  int64_t n_tokens, int32_t n_seqs, int32_t HQ, int32_t HKV, int32_t D,
                                  int32_t n_pages, int32_t page_size, int32_t max_pages, float scale, const void* z,
                                  void* o, void* workspace, size_t workspace_bytes, void* stream) {
    if (n_tokens < 0 || n_tokens > INT32_MAX || n_seqs < 0) return GDN_ERR_SHAPE;
    gdn_status st = check_heads(io_dtype, HQ, HKV, D);
    if (st != GDN_OK) return st;
    st = check_pages(n_pages, page_size, max_pages);
    if (st != GDN_OK) return st;
    if (!(scale - scale == 0.f)) return GDN_ERR_SHAPE;
    if (n_tokens == 0 || n_seqs == 0) return GDN_OK;
    if (!block_table || !kv_lens || !cu_seqlens) return GDN_ERR_NULL;
    const AttnArgs a{q, {k_cache, v_cache, block_table, kv_lens, n_pages, page_shift_of(page_size), max_pages},
                     cu_seqlens, 0, n_tokens, n_seqs, HQ, HKV, D, scale, z, o, io_dtype == GDN_BF16, workspace};
    return run_prefill(a, io_dtype, workspace, workspace_bytes, stream);
}

size_t gdn_attn_decode_workspace_bytes(int32_t B, int32_t HQ, int32_t HKV, int32_t D, gdn_dtype io_dtype) {
    return decode_bytes(B, HQ, HKV, D, io_dtype);
}

gdn_status gdn_attn_decode(const void* q, gdn_dtype io_dtype, const void* k_cache, const void* v_cache,
                           const int32_t* block_table, const int32_t* kv_lens, int32_t B, int32_t HQ, int32_t HKV,
                           int32_t D, int32_t n_pages, int32_t page_size, int32_t max_pages, float scale,
                           const void* z, void* o, void* workspace, size_t workspace_bytes, void* stream) {
    if (B < 0) return GDN_ERR_SHAPE;
    gdn_status st = check_heads(io_dtype, HQ, HKV, D);
    if (st != GDN_OK) return st;
    st = check_pages(n_pages, page_size, max_pages);
    if (st != GDN_OK) return st;
    if (!(scale - scale == 0.f)) return GDN_ERR_SHAPE;
    if (B == 0) return GDN_OK;
    if (!block_table || !kv_lens) return GDN_ERR_NULL;
    const AttnArgs a{q, {k_cache, v_cache, block_table, kv_lens, n_pages, page_shift_of(page_size), max_pages},
                     nullptr, 1, B, B, HQ, HKV, D, scale, z, o, io_dtype == GDN_BF16, workspace};
    st = check_attn(a, io_dtype, decode_bytes(B, HQ, HKV, D, io_dtype), workspace, workspace_bytes);
    if (st != GDN_OK) return st;
    return cuda_status(gdn::launch_attn_decode(a, (cudaStream_t)stream));
}

gdn_status gdn_attn_status(int32_t* device_error) {
    if (!device_error) return GDN_ERR_NULL;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_status(e);
    int32_t word = 0;
    for (auto read : {gdn::read_append_error, gdn::read_attn_cudacore_error, gdn::read_attn_decode_error,
                      gdn::read_attn_tc_error, gdn::read_attn_plan_error}) {
        int32_t w = 0;
        e = read(&w);
        if (e != cudaSuccess) return cuda_status(e);
        if (word == 0) word = w;
    }
    *device_error = word;
    return word ? GDN_ERR_DEVICE : GDN_OK;
}

}  // extern "C"
