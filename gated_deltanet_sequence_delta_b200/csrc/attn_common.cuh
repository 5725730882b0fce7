// attn_common.cuh -- declarations shared by the attention kernels' .cu files.
#pragma once

#include <atomic>

#include "gdn_internal.cuh"
#include "paged.cuh"

namespace gdn {

// The key-value cache as the kernels see it.  table null: no cache; keys and values are the
// packed (or dense) tensors k, v, indexed like the queries.
struct AttnKv {
    const void* k;              // [n_pages, page_size, HKV, D], or [tokens, HKV, D]
    const void* v;
    const int32_t* table;       // [n_seqs, max_pages]
    const int32_t* kv_lens;     // [n_seqs]
    int n_pages, page_shift, max_pages;
};

struct AttnArgs {
    const void* q;              // [n_tokens, HQ, D]
    AttnKv kv;
    const int32_t* cu;          // [n_seqs + 1], or null: T tokens per sequence
    int64_t T;                  // tokens per sequence (dense)
    int64_t n_tokens;
    int n_seqs, HQ, HKV, D;
    float scale;
    const void* z;              // output gate inputs [n_tokens, HQ, D], or null
    void* o;                    // [n_tokens, HQ, D]
    bool bf16;
    void* ws;                   // scratch
    // paged prompt pieces of at most this many (token, query head of a group) rows go to the kernel that
    // streams the pages past one m16 product (attn_decode.cu), the others to the tiles; 0: none do
    int short_rows;
};

struct AppendArgs {
    const void* q;              // may be null (with q_out)
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    const float* inv_freq;      // [rotary / 2]
    int rotary;                 // leading elements of a head that are rotated
    bool interleaved;
    const int32_t* cu;
    int64_t n_tokens;
    int n_seqs, HQ, HKV, D;
    void* q_out;
    void* k_cache;
    void* v_cache;
    const int32_t* table;
    const int32_t* kv_lens;
    int n_pages, page_shift, max_pages;
    bool bf16;
};

__device__ __forceinline__ SeqRows seq_rows(const AttnArgs& a, int n) {
    return seq_rows(a.cu, a.kv.kv_lens, n, a.T, a.n_tokens, (int64_t)a.kv.max_pages << a.kv.page_shift);
}

__device__ __forceinline__ bool short_piece(const AttnArgs& a, const SeqRows& r) {
    return a.short_rows > 0 && r.n_q > 0 && (int64_t)r.n_q * (a.HQ / a.HKV) <= a.short_rows;
}

// Scratch of the prompt attentions, built by the plan kernel and filled in by the main one.
// A tile is the work of one key-value head on a run of a sequence's rows.
struct PlanTile {
    int n, index;               // sequence, which of its tiles
    int q0, n_q, n_kv;          // the sequence's rows (seq_rows)
    int steps;                  // key steps of 128 (kept by the tensor-core path), at least 1
    int before;                 // units of the tiles before it in the list (split plans only)
    int pad;
};
struct AttnPlan {
    int32_t* counts;            // [0] tiles, [1] records to redo, [3] blocks that share the steps evenly (a split
                                // plan), or 0: whole tiles
    PlanTile* tiles;            // longest key range first
    int4* redo;                 // {sequence, key-value head, first row, rows} of that head's (token, query head) rows
    int4* desc;                 // split plans, [block]: {tile, key-value head, first, last block} of the one the block began
                                // inside, as the first that did; or tile = -1
    float2* part_ml;            // pieces of tiles that blocks share: [block][2][256] (maximum, sum), and
    float* part_o;              // outputs, [block][2][tile of 128 rows][D / 4][128][4]
    int max_tiles, max_redo;
    bool can_split;
    size_t bytes;
};
constexpr int kSplitGrid = 160;     // blocks that a split plan has room for
constexpr int kSplitRows = 256;
// A split plan counts work in units: a (tile, key-value head)'s steps and, in front of them, its own
// start and end (queries in, outputs out, a step's chain that nothing overlaps) as this many steps
// (2048 tokens, 16 heads over 4: 79 us at 0, 54 at 2, 49 at 3, 50 at 4, 52 at 6; 2 x 1500, 32 over 8: 161,
// 106, 90, 89, 92).
constexpr int kSplitItem = 4;
// (Rows of a bad table may be listed twice: never past the list's end.)
__device__ __forceinline__ void list_redo(const AttnPlan& plan, int n, int kvh, int row, int rows) {
    const int k = atomicAdd(&plan.counts[1], 1);
    if (k < plan.max_redo) plan.redo[k] = make_int4(n, kvh, row, rows);
}
// Tiles of `tile_rows` rows, `row_per_tok` rows a token; room for `redo` records a tile; split_heads > 0:
// a plan that may split tiles between blocks, that many key-value heads to a tile.
AttnPlan attn_plan(void* ws, int64_t n_tokens, int n_seqs, int redo, int row_per_tok, int tile_rows, int split_heads,
                   int D);
cudaError_t launch_attn_plan(const AttnArgs& a, const AttnPlan& p, int row_per_tok, int tile_rows, int grid,
                             cudaStream_t s);

// Launch with programmatic stream serialisation: the kernel may start while the one before it
// drains, and waits in griddepcontrol.wait before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*f)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, f, args...);
}

// Let a kernel use `bytes` of dynamic shared memory, once per device (`done`, a bit a device, is
// the kernel's own): the call costs as much as a third of a launch.
inline cudaError_t allow_smem(const void* f, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// out * sigmoid(z)
__device__ __forceinline__ float gate_out(float o, float z) { return o / (1.0f + expf(-z)); }
// The same for a result that is rounded to bf16: the special-function units' 2^x and reciprocal
// (a few 2^-23 each, against the rounding's 2^-8) without the division's fix-up.
__device__ __forceinline__ float gate_out_fast(float o, float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return o * r;
}

// Pieces that short_piece() names, against their pages; rows whose result is not finite are listed in
// the plan.  `ws` as the decode call's.
constexpr int kShortRows = 16;
cudaError_t launch_attn_short(const AttnArgs& a, const AttnPlan& plan, void* ws, cudaStream_t s);
cudaError_t launch_attn_append(const AppendArgs& a, cudaStream_t s);
cudaError_t launch_attn_cudacore(const AttnArgs& a, cudaStream_t s);
// bf16 on the tensor cores; the query heads of a group have to fit a tile's rows.
bool attn_tc_supported(int HQ, int HKV);
// 0: more sequences than the lists count.
size_t attn_tc_bytes(int64_t n_tokens, int n_seqs, int HQ, int HKV, int D);
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s);
// Redo the rows that the plan lists, on CUDA cores.
cudaError_t launch_attn_redo(const AttnArgs& a, const AttnPlan& p, cudaStream_t s);
cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s);
size_t attn_decode_bytes(int D);
size_t attn_cudacore_bytes(int64_t n_tokens, int n_seqs, int HQ, int HKV, int D);

// Read (and clear) the device word each file's kernels set on a bad table or an expired wait.
cudaError_t read_append_error(int32_t* out);
cudaError_t read_attn_cudacore_error(int32_t* out);
cudaError_t read_attn_decode_error(int32_t* out);
cudaError_t read_attn_tc_error(int32_t* out);
cudaError_t read_attn_plan_error(int32_t* out);

}  // namespace gdn
