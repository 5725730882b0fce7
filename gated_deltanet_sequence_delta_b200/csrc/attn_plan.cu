// attn_plan.cu -- the work list of the prompt attentions.  Lengths live on the device, so the list
// is made there, by one block, in front of the kernel that works it off.
//
// Every sequence's tiles, the longest key ranges first (blocks start in that order, so the short
// ones fill the end): a counting sort over kBuckets ranges of length.  The order inside a bucket
// varies from run to run and changes no result.
//
// Where there are few tiles and some are long (drafts or a prompt's last tokens over long pasts),
// whole tiles would leave most blocks idle or waiting for the longest.  The plan is then split:
// the tiles' steps of 128 keys are numbered through and every block takes an equal run of them.
// A (tile, key-value head)'s own start and end is counted as kSplitItem steps more: by steps alone the
// last blocks get many one-step tiles (2048 tokens, 16 heads over 4: 79 us, with it 50).
// The plan is split where the longest tile exceeds an even share by more than kSplitSlack units, about
// what writing and joining the pieces costs.  Split against whole at an excess of 101 units 69 against
// 187 us, 18: 56 / 71, 11: 34 / 46, 10: 50 / 55, 9: 50 / 50, 8: 64 / 60, none: 89 / 74.
#include "attn_common.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

__device__ int g_plan_error;

constexpr int kPlanThreads = 1024, kBuckets = 256;
constexpr int kSplitTiles = kPlanThreads;         // tiles that a split plan may list
constexpr int kSplitSlack = 8, kSplitMin = 4;     // units

// Tiles of a sequence in the list.  The sequences of a proper table have plan.max_tiles together at most.
// Those of a decreasing cu_seqlens may name rows over and over, in sum more than 32 bits count: a list that
// would be longer than its place is not made.
__device__ __forceinline__ int64_t tiles_of(const AttnArgs& a, const SeqRows& r, int per, int tile_rows) {
    return short_piece(a, r) ? 0 : ((int64_t)r.n_q * per + tile_rows - 1) / tile_rows;
}

// The list of at most kSplitTiles tiles, in a fixed order (a split tile's sums depend on it), with
// the units before each tile, and whether to split.  A tile a thread.
template <typename F>
__device__ void split_plan(const AttnArgs& a, const AttnPlan& plan, int per, int tile_rows, int grid, F keys_of) {
    __shared__ int s_start[kSplitTiles], s_steps[kSplitTiles], s_warp[kPlanThreads / 32], s_max;
    const int tid = threadIdx.x, lane = tid & 31;
    // the tiles before each sequence
    int mine = 0;
    if (tid < a.n_seqs) {
        const SeqRows r = seq_rows(a, tid);
        if (r.bad) atomicMax(&g_plan_error, r.bad);
        mine = (int)tiles_of(a, r, per, tile_rows);      // (within the 1024 that can_split allows, and so the sum)
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[tid >> 5] = incl;
    if (tid == 0) s_max = 0;
    __syncthreads();
    int base = 0, tiles = 0;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
        if (i < (tid >> 5)) base += s_warp[i];
        tiles += s_warp[i];
    }
    if (tiles > plan.max_tiles) tiles = 0;
    s_start[tid] = base + incl - mine;
    __syncthreads();
    // this thread's tile: the last sequence that starts at or before it and has tiles
    PlanTile t = {};
    if (tid < tiles) {
        int lo = 0, hi = a.n_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_start[mid] <= tid)
                lo = mid;
            else
                hi = mid - 1;
        }
        const SeqRows r = seq_rows(a, lo);
        t = PlanTile{lo, tid - s_start[lo], r.q0, r.n_q, r.n_kv, 0, 0, 0};
        t.steps = max((keys_of(r, t.index) + 127) / 128, 1);
        atomicMax(&s_max, t.steps);
    }
    s_steps[tid] = t.steps;
    __syncthreads();
    // its place: after the longer tiles, and the equal ones before it
    int rank = 0;
    int64_t total = 0;
    for (int j = 0; j < tiles; ++j) {
        const int w = s_steps[j];
        const bool first = w > t.steps || (w == t.steps && j < tid);
        rank += first;
        t.before += first ? w + kSplitItem : 0;
        total += w + kSplitItem;
    }
    if (tid < tiles) plan.tiles[rank] = t;
    if (tid == 0) {
        const int64_t units = total * a.HKV, share = (units + grid - 1) / grid;
        int blocks = 0;
        if (s_max + kSplitItem > share + kSplitSlack && total <= INT32_MAX / 2)      // (`before` is 32 bits)
            blocks = (int)min((int64_t)grid, max(units / kSplitMin, (int64_t)1));
        plan.counts[0] = tiles;
        plan.counts[1] = 0;
        plan.counts[3] = blocks;
    }
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(AttnArgs a, AttnPlan plan, int per, int tile_rows,
                                                                 int grid) {
    __shared__ int s_count[kBuckets];
    __shared__ int s_max;
    __shared__ unsigned long long s_tiles;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < kBuckets; i += kPlanThreads) s_count[i] = 0;
    if (tid == 0) {
        s_max = 1;
        s_tiles = 0;
    }
    __syncthreads();
    tc::grid_dependency_sync();
    auto keys_of = [&](const SeqRows& r, int t) {          // keys that the tile's last row sees
        const int64_t last = min(((int64_t)t + 1) * tile_rows, (int64_t)r.n_q * per) - 1;
        return max(r.n_kv - r.n_q + (int)(last / per) + 1, 0);
    };
    if (plan.can_split) {
        split_plan(a, plan, per, tile_rows, grid, keys_of);
        return;
    }
    int mx = 1;
    int64_t all = 0;
    for (int n = tid; n < a.n_seqs; n += kPlanThreads) {
        const SeqRows r = seq_rows(a, n);
        if (r.bad) atomicMax(&g_plan_error, r.bad);
        mx = max(mx, r.n_kv);
        all += tiles_of(a, r, per, tile_rows);
    }
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane == 0) atomicAdd(&s_tiles, (unsigned long long)all);
    atomicMax(&s_max, mx);
    __syncthreads();
    if (s_tiles > (unsigned long long)plan.max_tiles) {
        if (tid == 0) plan.counts[0] = plan.counts[1] = plan.counts[3] = 0;
        return;
    }
    const int width = (s_max - 1) / kBuckets + 1;
    // a sequence per warp, a tile per lane
    for (int pass = 0; pass < 2; ++pass) {
        for (int n = tid >> 5; n < a.n_seqs; n += kPlanThreads / 32) {
            const SeqRows r = seq_rows(a, n);
            const int tiles = (int)tiles_of(a, r, per, tile_rows);
            for (int t = lane; t < tiles; t += 32) {
                const int keys = keys_of(r, t);
                const int at = atomicAdd(&s_count[kBuckets - 1 - min(keys / width, kBuckets - 1)], 1);
                // (tables that change under the call: never past the list's end)
                if (pass == 1 && at < plan.max_tiles)
                    plan.tiles[at] = PlanTile{n, t, r.q0, r.n_q, r.n_kv, max((keys + 127) / 128, 1), 0, 0};
            }
        }
        __syncthreads();
        if (pass == 0 && tid < 32) {      // exclusive sums of the buckets, kBuckets / 32 a lane
            constexpr int E = kBuckets / 32;
            int v[E], sum = 0;
            for (int e = 0; e < E; ++e) {
                v[e] = s_count[tid * E + e];
                sum += v[e];
            }
            int incl = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (tid >= o) incl += y;
            }
            int base = incl - sum;
            for (int e = 0; e < E; ++e) {
                s_count[tid * E + e] = base;
                base += v[e];
            }
            if (tid == 31) {
                plan.counts[0] = min(incl, plan.max_tiles);
                plan.counts[1] = 0;
                plan.counts[3] = 0;
            }
        }
        __syncthreads();
    }
}

}  // namespace

AttnPlan attn_plan(void* ws, int64_t n_tokens, int n_seqs, int redo, int row_per_tok, int tile_rows, int split_heads,
                   int D) {
    AttnPlan p;
    const int64_t tiles = (n_tokens * row_per_tok + tile_rows - 1) / tile_rows + n_seqs;
    uint8_t* b = static_cast<uint8_t*>(ws);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    p.max_tiles = (int)tiles;
    p.max_redo = (int)(tiles * redo);
    p.counts = reinterpret_cast<int32_t*>(b);
    size_t at = kStatusBytes;
    p.tiles = reinterpret_cast<PlanTile*>(b + at);
    at += up((size_t)tiles * sizeof(PlanTile));
    p.redo = reinterpret_cast<int4*>(b + at);
    at += up((size_t)tiles * redo * sizeof(int4));
    // with more tiles than this, whole ones keep the blocks evenly busy
    p.can_split = split_heads > 0 && tiles * split_heads <= 4 * kSplitGrid && tiles <= kSplitTiles;
    p.desc = reinterpret_cast<int4*>(b + at);
    if (p.can_split) at += up(kSplitGrid * sizeof(int4));
    p.part_ml = reinterpret_cast<float2*>(b + at);
    if (p.can_split) at += (size_t)kSplitGrid * 2 * kSplitRows * sizeof(float2);
    p.part_o = reinterpret_cast<float*>(b + at);
    if (p.can_split) at += (size_t)kSplitGrid * 2 * kSplitRows * D * sizeof(float);
    p.bytes = at;
    return p;
}

cudaError_t launch_attn_plan(const AttnArgs& a, const AttnPlan& p, int row_per_tok, int tile_rows, int grid,
                             cudaStream_t s) {
    const cudaError_t e = launch_pdl(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, p, row_per_tok, tile_rows,
                                     grid);
    if (e == cudaSuccess) count_launch();
    return e;
}

cudaError_t read_attn_plan_error(int32_t* out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_plan_error, sizeof(int32_t));
    if (e == cudaSuccess && *out != 0) {
        const int32_t zero = 0;
        e = cudaMemcpyToSymbol(g_plan_error, &zero, sizeof(int32_t));
    }
    return e;
}

}  // namespace gdn
