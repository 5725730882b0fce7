// attn_prefill_tc.cu -- causal grouped attention of prompts on the tensor cores (bf16).
//
//   S = scale Q K^T,  P = e^{S - m} (0 where a row does not see a key),  O = P V / rowsum(P)
//
// in one pass over the keys with a running reference m per row.  FLOPs: 4 D per (row, key) pair,
// 2 D x 2 products; bound by the tensor cores and, at D = 64, by the exponentials: an SM takes
// 16 of them a clock in its special-function units, so the 128 x 128 weights of a step cost 1024
// clocks there against 1024 (D = 128) or 512 (D = 64) of the two products.
//
// Rows.  A tile is 128 rows, the (token, query head of the group) pairs of one key-value head:
// 128 / G tokens by G heads, so that the group shares every key and value that is staged and
// the diagonal's waste shrinks with G (rows left over where G does not divide 128 are idle).  A
// block takes two consecutive tiles, A and B, against the same keys: while the softmax of one
// runs, the tensor cores work for the other.  Blocks are persistent, so that an item's first
// loads and scores run under the last item's outputs.
//
// Roles (12 warps, one block per SM):
//   warps 0-3, 4-7   softmax of tile A, of tile B: a thread owns a row (TMEM lane), takes its 128
//                    scores into registers, forms the weights, writes them as bf16
//   warps 8, 9       issue the MMAs of tile A, of tile B: per step  S = Q K',  O += P V  (K' the
//                    next step's keys); two warps, so that neither tile's products wait behind
//                    the other's softmax
//   warps 10, 11     TMA: the work items, their queries and the keys; the values.  Keys and values
//                    go through one ring
// TMEM, 512 columns: S 128, P_A and P_B 64 each, O_A and O_B D each.  A tile's scores of the next
// step are formed while its softmax works on the last ones, so that the products stay off that
// chain; at D = 128 this leaves room for one S, which the tiles use in turn (it is free again
// once its softmax warps have read it), at D = 64 for one each.
//
// The reference m need not be the running maximum, only near it: weights up to 2^15 lose nothing in
// fp32 sums and products, nor in bf16's range.  So a step first forms its weights against m as it
// is, without looking for a maximum, and keeps them unless a row's sum exceeds 2^15; only then (and
// where a mask cuts the step) are the maxima found, m moved where it has been passed by more than
// 2^8, and the accumulated O rescaled in tensor memory: a row's first steps.  The weights are rounded
// to bf16 for the product (half a step, 2^-8 relative, each); their sum is taken before the rounding.
//
// Measured, bf16: one prompt of 32K tokens, 16 heads over 4 of 128: 3.4 ms in short runs (1.28 PFLOP/s,
// 0.76 of the matrix rate), 3.8-4.0 ms in long ones, where the power limit holds the clock at 1.63 GHz
// (0.79 of the sustained matrix rate); 75K packed tokens, gated: 3.4-3.8 ms, 3.8-4.0 in long runs; pieces
// over contexts to 24K, gated: 1.6 ms (1.8); 18 to 40 tokens over 13K in pages of 16: 90-92 us.  16 heads
// over 4 of 64: 8K tokens 224 us, 32K 2.86 ms.
//
// Masked weights are exact zeros, but 0 * v is not 0 where v is infinite or NaN.  Values past
// the last key that any row of the block sees are cleared in shared memory, by each tile before its
// product reads them; a value inside the diagonal that is not finite shows in the outputs, whose
// tile is then put on a list that the CUDA-core kernel, which leaves masked places out of its sums,
// does again.
#include "attn_common.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

using bf16 = __nv_bfloat16;

__device__ int g_attn_tc_error;

constexpr int kThreads = 384;
// Registers: 384 threads launch with 168 each; the two softmax warpgroups take 216, the third
// keeps 72 (2 x 216 + 72 = 3 x 168).
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
constexpr int kRows = 128, kKeys = 128;
constexpr int kItems = 8;                // work items known ahead
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;            // growth of the maximum (log2) that moves the reference,
constexpr float kGrowSum = 32768.0f;     // where it is looked at: when a step's weights sum to more than this

template <int D>
struct Cfg {
    static constexpr int kHalves = D / 64;                       // 128-byte column blocks
    static constexpr int kTile = 128 * D * 2;                    // bytes of 128 rows
    static constexpr int kHalf = 128 * 128;                      // bytes of one column block
    static constexpr int kRing = D == 128 ? 5 : 8;               // key / value tiles
    static constexpr int kSmem = (2 + kRing) * kTile + 1024;
    static constexpr bool kOneS = D == 128;                      // one S for both tiles
    // TMEM columns
    __device__ static constexpr int s_col(int x) { return kOneS ? 0 : x * 128; }
    __device__ static constexpr int p_col(int x) { return (kOneS ? 128 : 256) + x * 64; }
    __device__ static constexpr int o_col(int x) { return 512 - 2 * D + x * D; }
};

// Two floats side by side, and the FMA pipes' two-wide operations on them.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float exp2_sfu(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A row's weights 2^(s sc - base) as bf16 in tensor memory (keys 2j, 2j + 1 in column j); returns
// their sum.  `free` is called before the first write.  MASKED: keys past `last` weigh exactly 0.
// All weights go through the special-function units, which keep NaN and infinities: forming an eighth
// of them on the FMA pipes by a cubic (2^f on [-1/2, 1/2], the integer part added to the exponent, the
// argument bound on both sides) takes as long or longer: 227 against 224 us for 8K tokens, 16 heads over 4
// of 64, 2.94 / 2.86 ms for 32K; of 128, 3.48 / 3.43 ms.
template <bool MASKED, typename F>
__device__ __forceinline__ float weights(const float (&s)[128], float sc, float base, int last, uint32_t tp, F free) {
    const uint64_t sc2 = pack2(sc, sc), nb2 = pack2(-base, -base);
    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            float e0, e1;
            unpack2(fma2(pack2(s[c + j], s[c + j + 1]), sc2, nb2), e0, e1);
            if (MASKED) {
                e0 = c + j > last ? 0.f : exp2_sfu(e0);
                e1 = c + j + 1 > last ? 0.f : exp2_sfu(e1);
            } else {
                e0 = exp2_sfu(e0);
                e1 = exp2_sfu(e1);
            }
            sum[(j >> 1) & 3] = add2(sum[(j >> 1) & 3], pack2(e0, e1));
            p[j / 2] = pack_bf16(e0, e1);
        }
        if (c == 0) free();
        tc::tmem_st16_raw(tp + c / 2, p);
    }
    float a, b;
    unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
    return a + b;
}

// One item of a block's work: tiles A and B of a (sequence, tile pair, key-value head), or the
// steps s0 .. s1 - 1 of it.
struct Item {
    int n, kvh, q0, n_q, n_kv;
    int tok;                   // first token of A; B follows `tokens` later
    int s0, s1;
    int slot;                  // where a piece's sums go, -1: the item is whole; -2: no more items
    __device__ __forceinline__ int past() const { return n_kv - n_q; }
    // of tile x: tokens it has (0: no tile), keys its last row sees, steps of 128 keys of this item
    __device__ __forceinline__ int ntok(int x, int tokens) const { return max(min(tokens, n_q - tok - x * tokens), 0); }
    __device__ __forceinline__ int end(int x, int tokens) const {
        const int k = ntok(x, tokens);
        return k > 0 ? max(past() + tok + x * tokens + k, 0) : 0;
    }
    __device__ __forceinline__ int steps(int x, int tokens) const {
        return max(min((end(x, tokens) + kKeys - 1) / kKeys, s1) - s0, 0);
    }
    __device__ __forceinline__ int total(int tokens) const { return max(steps(0, tokens), steps(1, tokens)); }
    // the tile of its first step
    __device__ __forceinline__ int first(int tokens) const { return steps(0, tokens) > 0 ? 0 : 1; }
};

// The items of this block, in order.  Warp-wide.
struct ItemSource {
    int tiles, shared, k;
    int64_t at, stop;
    __device__ __forceinline__ ItemSource(const AttnArgs& a, const AttnPlan& plan, int tokens) {
        tiles = plan.counts[0];
        shared = plan.counts[3];
        k = 0;
        at = stop = 0;
        if (shared == 0 || (int)blockIdx.x >= shared) return;
        // an even share of all units, tile by tile, key-value head by key-value head
        const int lane = threadIdx.x & 31;
        const PlanTile end = plan.tiles[tiles - 1];
        const int64_t N = (int64_t)(end.before + end.steps + kSplitItem) * a.HKV;
        at = N * blockIdx.x / shared;
        stop = N * (blockIdx.x + 1) / shared;
        for (int b = 0; b < tiles; b += 32) {          // the tile that holds unit `at`
            const bool in = b + lane < tiles && (int64_t)plan.tiles[b + lane].before * a.HKV <= at;
            const unsigned m = __ballot_sync(0xffffffffu, in);
            if (m) k = b + 31 - __clz(m);
        }
        if (lane == 0 && blockIdx.x > 0) {             // for the join
            const PlanTile t = plan.tiles[k];
            const int w = t.steps + kSplitItem, h = (int)((at - (int64_t)t.before * a.HKV) / w);
            // the (tile, head)'s blocks: the first is the last one that begins at or before its
            // first step (no share is empty: there are at least as many units as blocks)
            const int64_t t0 = (int64_t)t.before * a.HKV + (int64_t)h * w + kSplitItem;
            const int c0 = (int)(((t0 + 1) * shared - 1) / N), c1 = (int)(((t0 + t.steps) * shared - 1) / N);
            plan.desc[blockIdx.x] =
                at > t0 && (int)blockIdx.x == c0 + 1 ? make_int4(k, h, c0, c1) : make_int4(-1, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void next(const AttnArgs& a, const AttnPlan& plan, int tokens, Item& it) {
        const int G = a.HQ / a.HKV, lane = threadIdx.x & 31;
        while (true) {
            if (shared == 0) {
                // whole tiles: the list runs from long to short; blocks take it forwards and
                // backwards in turn, which evens out their sums
                const int64_t i = (int64_t)k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                if (i >= (int64_t)tiles * a.HKV) break;
                ++k;
                const PlanTile t = plan.tiles[i / a.HKV];
                it = Item{t.n, (int)(i % a.HKV), t.q0, t.n_q, t.n_kv, t.index * 2 * tokens, 0, t.steps, -1};
            } else {
                if (at >= stop) break;
                const PlanTile t = plan.tiles[k];
                const int64_t o = at - (int64_t)t.before * a.HKV;
                const int w = t.steps + kSplitItem, h = (int)(o / w);
                if (h >= a.HKV) {
                    ++k;
                    continue;
                }
                const int s0 = (int)(o - (int64_t)h * w) - kSplitItem;
                if (s0 < 0) {                              // to its first step
                    at -= s0;
                    continue;
                }
                const int s1 = (int)min((int64_t)t.steps, s0 + stop - at);
                it = Item{t.n, h, t.q0, t.n_q, t.n_kv, t.index * 2 * tokens, s0, s1,
                          s0 == 0 && s1 == t.steps ? -1 : (int)blockIdx.x * 2 + (s0 == 0 ? 1 : 0)};
                at += s1 - s0;
            }
            if (it.total(tokens) > 0) return;
            // no row of the tile sees a key: the CUDA-core kernel writes its zeros
            for (int row = lane * 64; row < 2 * tokens * G; row += 32 * 64)
                list_redo(plan, it.n, it.kvh, it.tok * G + row, min(64, 2 * tokens * G - row));
        }
        it.slot = -2;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(const __grid_constant__ CUtensorMap tq,
                                                                   const __grid_constant__ CUtensorMap tk,
                                                                   const __grid_constant__ CUtensorMap tv,
                                                                   const __grid_constant__ CUtensorMap tz,
                                                                   const __grid_constant__ CUtensorMap to_map, AttnArgs a,
                                                                   AttnPlan plan, int tokens, int box_rows) {
    using C = Cfg<D>;
    constexpr int S = C::kRing;
    extern __shared__ uint8_t smem_raw[];
    // q_full, q_used, z_full, q_empty: a tile's place for queries holds them, is done with, holds the
    // gate's inputs (or is free for the outputs), is free; staged: the outputs are in it
    __shared__ __align__(8) uint64_t q_full[2], q_used[2], z_full[2], staged[2], q_empty[2];
    // s_full: scores formed; turn: S is this tile's to fill; p_full: weights written; pv_done: their
    // product has read them; v_last: the item's last values are there
    __shared__ __align__(8) uint64_t s_full[2], turn[2], p_full[2], pv_done[2], v_last[2];
    __shared__ __align__(8) uint64_t kv_full[S], kv_empty[S], item_full[kItems], item_empty[kItems], drain[2];
    __shared__ Item s_item[kItems];
    __shared__ uint32_t s_tmem;
    __shared__ int s_timeout;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* q_smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* ring = q_smem + 2 * C::kTile;
    const int G = a.HQ / a.HKV;

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            tc::mbar_init(&kv_full[i], 1);
            tc::mbar_init(&kv_empty[i], 2);
        }
        for (int x = 0; x < 2; ++x) {
            tc::mbar_init(&q_full[x], 1);
            tc::mbar_init(&q_empty[x], 4);
            tc::mbar_init(&q_used[x], 1);
            tc::mbar_init(&z_full[x], 1);
            tc::mbar_init(&staged[x], 4);
            tc::mbar_init(&s_full[x], 1);
            tc::mbar_init(&turn[x], 4);
            tc::mbar_init(&p_full[x], 4);
            tc::mbar_init(&pv_done[x], 1);
            tc::mbar_init(&v_last[x], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            tc::mbar_init(&item_full[i], 1);
            tc::mbar_init(&item_empty[i], 11);
        }
        tc::mbar_init(&drain[0], 1);
        tc::mbar_init(&drain[1], 1);
        tc::fence_mbar_init();
        s_timeout = 0;
    }
    if (warp == 8) {
        tc::tmem_alloc(&s_tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;
    tc::grid_dependency_sync();          // the plan is ready, and what ran before has left o alone

    // the item ring's reader side: item r, or slot -2 past the last one (or after an expired wait)
    auto item_at = [&](int r, bool& ok) {
        Item it;
        if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&item_full[r % kItems], (uint32_t)(r / kItems) & 1u));
        it = s_item[r % kItems];
        if (!ok) it.slot = -2;
        return it;
    };
    auto item_done = [&](int r) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&item_empty[r % kItems]);
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp < 10) {
            // ---- products of tile x ---------------------------------------------------------
            // (the whole warp walks the loop, one elected lane issues)
            const int x = warp - 8;
            const uint32_t neg = a.scale < 0.f ? 1u << 13 : 0u;        // -Q: scores of a negative scale
            const uint32_t id_s = tc::idesc_bf16(128, kKeys, 0, 0) | neg, id_o = tc::idesc_bf16(128, D, 0, 1);
            const uint64_t qd = tc::desc_sw128(tc::smem_u32(q_smem + x * C::kTile), 0, 1024);
            const uint64_t kd = tc::desc_sw128(tc::smem_u32(ring), 0, 1024);
            const uint64_t vd = tc::desc_sw128(tc::smem_u32(ring), C::kHalf, 1024);
            bool ok = true;
            int t0 = 0, items = 0, loads = 0, mine = 0;                // ring tiles, items, queries and steps before this item
            int turns = -1;                                            // phases of turn[x] taken
            auto wait = [&](uint64_t* bar, int phase) {
                if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait_short(bar, (uint32_t)phase & 1u));
            };
            auto wait_kv = [&](int t) { wait(&kv_full[t % S], t / S); };
            for (int r = 0; ok; ++r) {
                const Item it = item_at(r, ok);
                item_done(r);
                if (it.slot == -2) break;
                const int steps = it.steps(x, tokens), total = it.total(tokens);
                if (items == 0 && C::kOneS && it.first(tokens) != x) turns = 0;
                if (steps > 0) wait(&q_full[x], loads++);
                ++items;
                for (int i = -1; i < total && ok; ++i) {               // S(i + 1), then O += P(i) V(i)
                    if (i + 1 < total) {
                        const int t = i < 0 ? t0 : t0 + 2 * i + 1;     // ring tile of K(i + 1)
                        wait_kv(t);
                        if (i + 1 < steps) {
                            // S is ours once its last user has read it (the first time it is free)
                            if (turns >= 0) wait(&turn[x], turns);
                            ++turns;
                            tc::tc_fence_after();
                            if (ok && tc::elect_one()) {
                                const uint64_t k_off = (uint64_t)((t % S) * (C::kTile >> 4));
#pragma unroll
                                for (int k = 0; k < D / 16; ++k) {
                                    const uint32_t off = ((k >> 2) * C::kHalf + (k & 3) * 32) >> 4;
                                    tc::mma_bf16(tmem + C::s_col(x), qd + off, kd + k_off + off, id_s, k > 0);
                                }
                                tc::mma_commit(&s_full[x]);
                                tc::mma_commit(&kv_empty[t % S]);
                                if (i + 2 == steps) tc::mma_commit(&q_used[x]);
                            }
                        } else if (ok && lane == 0) {
                            tc::mbar_arrive(&kv_empty[t % S]);         // a tile of keys that only the other tile takes
                        }
                        __syncwarp();
                    }
                    const int t = t0 + (i + 1 < total ? 2 * i + 2 : 2 * i + 1);       // ring tile of V(i)
                    if (i >= 0) wait_kv(t);
                    if (i >= 0 && i < steps) {
                        if (i + 1 == total && ok && lane == 0) tc::mbar_arrive(&v_last[x]);
                        __syncwarp();
                        wait(&p_full[x], mine + i);
                        tc::tc_fence_after();
                        if (ok && tc::elect_one()) {
                            const uint64_t v_off = (uint64_t)((t % S) * (C::kTile >> 4));
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)
                                tc::mma_bf16_ts(tmem + C::o_col(x), tmem + C::p_col(x) + k * 8, vd + v_off + k * 128, id_o,
                                                i > 0 || k > 0);
                            tc::mma_commit(&pv_done[x]);
                            tc::mma_commit(&kv_empty[t % S]);
                        }
                    } else if (i >= 0 && ok && lane == 0) {
                        tc::mbar_arrive(&kv_empty[t % S]);
                    }
                    __syncwarp();
                }
                t0 += 2 * total;
                mine += steps;
            }
            // every arrival of the commits above has landed before the block leaves
            if (tc::elect_one()) tc::mma_commit(&drain[x]);
            __syncwarp();
            if (!tc::mbar_wait_short(&drain[x], 0) || !ok) s_timeout = 1;
        } else {
            // ---- loads: warp 10 the items, queries and keys, warp 11 the values ------------------
            // The ring takes K(0), K(1), V(0), K(2), V(1), ..., V(last) of an item.  (Its slots pass
            // between the two warps; what was in one two turns ago is long used by then, since the
            // products use the tiles in order.)
            const bool is_v = warp == 11;
            const CUtensorMap* map = is_v ? &tv : &tk;
            const int boxes = kKeys / box_rows;
            const int lg = lane / C::kHalves, lh = lane % C::kHalves;  // this lane's box, its column block
            const int none = (int)((int64_t)a.kv.n_pages << a.kv.page_shift);
            const bool paged = a.kv.table != nullptr && lg < boxes;
            bool ok = true;
            int t0 = 0;                                                // ring tiles before this item
            // This lane's page of a step, read ahead: a copy must not wait for its address.
            auto entry = [&](const Item& it, int step) {
                const int pos = (it.s0 + step) * kKeys + lg * box_rows;
                return paged && pos < it.n_kv ? a.kv.table[(int64_t)it.n * a.kv.max_pages + (pos >> a.kv.page_shift)] : 0;
            };
            auto load = [&](const Item& it, int step, int t, int page) {
                const int pos = (it.s0 + step) * kKeys + lg * box_rows, slot = t % S;
                int row = it.q0 + pos;
                if (paged) {
                    row = none;                                        // past the context or the cache: zero fill
                    if (pos < it.n_kv) {
                        if (page >= 0 && page < a.kv.n_pages)
                            row = (page << a.kv.page_shift) + (pos & ((1 << a.kv.page_shift) - 1));
                        else
                            atomicMax(&g_attn_tc_error, GDN_DEVERR_PAGE);
                    }
                }
                if (t >= S) ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&kv_empty[slot], (uint32_t)((t / S) & 1) ^ 1u));
                if (!ok) return;
                if (lane == 0) tc::mbar_expect_tx(&kv_full[slot], C::kTile);
                __syncwarp();
                if (lg < boxes)
                    tc::tma_load_3d(ring + slot * C::kTile + lh * C::kHalf + lg * box_rows * 128, map, &kv_full[slot], lh * 64,
                                    it.kvh, row);
            };
            int uses[2] = {0, 0};                                      // queries of each tile loaded (or used up) so far
            if (is_v) {
                for (int r = 0; ok; ++r) {
                    const Item it = item_at(r, ok);
                    item_done(r);
                    if (it.slot == -2) break;
                    const int total = it.total(tokens);
                    int page = entry(it, 0);
                    for (int j = 0; j < total && ok; ++j) {
                        const int after = entry(it, j + 1);
                        load(it, j, t0 + (j + 1 < total ? 2 * j + 2 : 2 * j + 1), page);
                        page = after;
                    }
                    t0 += 2 * total;
                    // a tile whose queries have done their part: their place takes the gate's inputs, and
                    // then the outputs on their way to memory
                    for (int x = 0; x < 2 && ok; ++x) {
                        if (it.steps(x, tokens) == 0) continue;
                        ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&q_used[x], (uint32_t)uses[x] & 1u));
                        ++uses[x];
                        if (ok && tc::elect_one()) {
                            if (a.z && it.slot < 0) {
                                tc::mbar_expect_tx(&z_full[x], (uint32_t)(C::kHalves * tokens * G * 128));
                                for (int h = 0; h < C::kHalves; ++h)
                                    tc::tma_load_3d(q_smem + x * C::kTile + h * C::kHalf, &tz, &z_full[x], h * 64, it.kvh * G,
                                                    it.q0 + it.tok + x * tokens);
                            } else {
                                tc::mbar_arrive(&z_full[x]);
                            }
                        }
                        __syncwarp();
                    }
                }
            } else {
                ItemSource src(a, plan, tokens);
                Item it, ahead;
                int r = 0;
                auto put = [&](const Item& x) {                        // to the other roles
                    if (r >= kItems) ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&item_empty[r % kItems], (uint32_t)(r / kItems - 1) & 1u));
                    if (ok && lane == 0) {
                        s_item[r % kItems] = x;
                        tc::mbar_arrive(&item_full[r % kItems]);
                    }
                    __syncwarp();
                    ++r;
                };
                src.next(a, plan, tokens, it);
                put(it);
                while (ok && it.slot != -2) {
                    const int total = it.total(tokens);
                    int page = entry(it, 0);
                    for (int j = 0; j < total && ok; ++j) {
                        const int after = entry(it, j + 1);
                        load(it, j, t0 + (j == 0 ? 0 : 2 * j - 1), page);
                        page = after;
                        if (j > 0 || !ok) continue;
                        // with the first keys, the queries, and the next item for everyone
                        for (int x = 0; x < 2 && ok; ++x) {
                            if (it.steps(x, tokens) == 0) continue;
                            if (uses[x] > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&q_empty[x], (uint32_t)(uses[x] - 1) & 1u));
                            ++uses[x];
                            if (ok && tc::elect_one()) {
                                tc::mbar_expect_tx(&q_full[x], (uint32_t)(C::kHalves * tokens * G * 128));
                                for (int h = 0; h < C::kHalves; ++h)
                                    tc::tma_load_3d(q_smem + x * C::kTile + h * C::kHalf, &tq, &q_full[x], h * 64, it.kvh * G,
                                                    it.q0 + it.tok + x * tokens);
                            }
                            __syncwarp();
                        }
                        src.next(a, plan, tokens, ahead);
                        put(ahead);
                    }
                    t0 += 2 * total;
                    it = ahead;
                }
            }
            if (!ok) {       // an expired wait: give the copies under way time to land
                if (lane == 0) s_timeout = 1;
                for (int i = 0; i < S; ++i) tc::mbar_wait_short(&kv_full[i], 0, 1000000);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---- softmax: thread = row ---------------------------------------------------------
        const int x = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const int tok = row / G, g = row - tok * G;
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;         // TMEM lane 32 (warp % 4)
        const uint32_t ts = tmem + lane_base + C::s_col(x), tp = tmem + lane_base + C::p_col(x),
                       to = tmem + lane_base + C::o_col(x);
        const float sc = fabsf(a.scale) * kLog2e;
        bool ok = true;
        int t0 = 0, done = 0, lasts = 0;                               // ring tiles, steps and last steps before this item
        int outs = 0, stages = 0;                                      // outputs before it, phases of staged[x]
        for (int r = 0; ok; ++r) {
            Item it = item_at(r, ok);
            if (it.slot == -2) break;
            const int steps = it.steps(x, tokens), other = it.steps(x ^ 1, tokens), total = max(steps, other);
            // last key this row sees (idle rows: no mask; nothing of them is kept); keys are
            // counted from the item's first step
            const int first_key = it.s0 * kKeys;
            const int lim = tok < it.ntok(x, tokens) ? it.past() + it.tok + x * tokens + tok - first_key : INT32_MAX;
            // The first of the values past the item's last key, for a tile that takes the last step.  Each
            // tile clears them for its own product, which waits for its own weights only: the second one's
            // zeros meet zeros, and are over before its product gives the values' place back.  (Clearing
            // once, with a barrier between the tiles, costs 1 to 4 percent of a long prompt's time.)
            const int clear_from = steps == total ? max(it.end(0, tokens), it.end(1, tokens)) - first_key : INT32_MAX;
            float m = -INFINITY, l = 0.f;
            bool finite = true;
            for (int i = 0; i < steps; ++i) {
                ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&s_full[x], (uint32_t)(done + i) & 1u));
                if (!ok) break;
                tc::tc_fence_after();
                float s[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) tc::tmem_ld32_raw(ts + c, reinterpret_cast<uint32_t*>(s) + c);
                tc::tmem_wait_ld();
                tc::tc_fence_before();
                __syncwarp();
                // S goes to the tile whose step comes next, A(0) B(0) A(1) ...: each MMA warp waits for
                // every phase of its own barrier, one a turn
                int next = x;
                if (C::kOneS) {
                    const bool them = x == 0 ? i < other : i + 1 < other;
                    next = them ? x ^ 1 : x;
                    if (!them && i + 1 == steps) {
                        const Item after = item_at(r + 1, ok);
                        next = after.slot == -2 ? -1 : after.first(tokens);
                    }
                }
                if (lane == 0 && next >= 0) tc::mbar_arrive(&turn[next]);
                const int j0 = i * kKeys;
                // Later steps that every row sees whole: the weights against the reference as it is.
                // They stand if no row's sum says that it should have moved.
                const bool masked = __any_sync(0xffffffffu, j0 + kKeys - 1 > lim || (m == -INFINITY && lim != INT32_MAX));
                auto free = [&] {                        // the last step's product has read P
                    if (i > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&pv_done[x], (uint32_t)(done + i - 1) & 1u));
                    tc::tc_fence_after();
                };
                if (clear_from - j0 < kKeys) {
                    // Values that no row of the block sees may be anything: clear them, every warp its
                    // share, whatever rows it has.  (The MMA warp, which sees every copy land in turn,
                    // tells when they are there.)
                    const int slot = (t0 + 2 * total - 1) % S;                // the item's last values
                    ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&v_last[x], (uint32_t)lasts & 1u));
                    if (!ok) break;
                    uint8_t* v = ring + slot * C::kTile;
                    const int first = clear_from - j0;
                    for (int e = row; e < (kKeys - first) * 8 * C::kHalves; e += 128) {
                        const int vr = first + e / (8 * C::kHalves), c = e % (8 * C::kHalves);
                        *reinterpret_cast<uint4*>(v + (c >> 3) * C::kHalf + vr * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_async_smem();
                }
                bool stand = false;
                if (!masked) {
                    const float sum = weights<false>(s, sc, m, 0, tp, free);
                    stand = !__any_sync(0xffffffffu, !(sum <= kGrowSum) && lim != INT32_MAX);
                    if (stand) l += sum;
                }
                if (!ok) break;
                if (!stand) {
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (j0 + j > lim) s[j] = -INFINITY;
                    float mx = max3(s[0], s[1], s[2]), mx1 = max3(s[3], s[4], s[5]), mx2 = max3(s[6], s[7], s[8]),
                          mx3 = max3(s[9], s[10], s[11]);
#pragma unroll
                    for (int j = 12; j < 124; j += 8) {
                        mx = max3(mx, s[j], s[j + 1]);
                        mx1 = max3(mx1, s[j + 2], s[j + 3]);
                        mx2 = max3(mx2, s[j + 4], s[j + 5]);
                        mx3 = max3(mx3, s[j + 6], s[j + 7]);
                    }
                    mx = max3(mx, s[124], s[125]);
                    mx1 = max3(mx1, s[126], s[127]);
                    mx = max3(mx, mx1, fmaxf(mx2, mx3)) * sc;
                    if (!(mx == mx)) mx = INFINITY;         // (-inf * 0: nothing seen, or scale 0 and infinite scores)
                    const bool none = lim < j0;              // no key of this step is seen: m and l stay
                    if (none) mx = -INFINITY;
                    const bool move = mx > m + kGrow || (m == -INFINITY && !none);
                    if (move && mx == -INFINITY) finite = false;      // every key seen so far scores -inf
                    if (__any_sync(0xffffffffu, move)) {
                        const float alpha = move && m != -INFINITY ? exp2_sfu(m - mx) : 1.f;
                        if (move) {
                            l *= alpha;
                            m = mx;
                        }
                        if (i > 0) {
                            ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&pv_done[x], (uint32_t)(done + i - 1) & 1u));
                            if (!ok) break;
                            tc::tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                float o[16];
                                tc::tmem_ld16(to + c, o);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] *= alpha;
                                tc::tmem_st16_raw(to + c, reinterpret_cast<uint32_t*>(o));
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.f : m;
                    l += weights<true>(s, sc, base, lim - j0, tp, free);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (!ok) break;
                if (lane == 0) tc::mbar_arrive(&p_full[x]);
            }
            if (!ok) break;
            it = s_item[r % kItems];                      // (again: not kept in registers over the loop)
            item_done(r);
            const int ntok = it.ntok(x, tokens);
            const bool live = tok < ntok;
            const int64_t at = (((int64_t)it.q0 + it.tok + x * tokens + tok) * a.HQ + it.kvh * G + g) * D;
            if (steps > 0) {
                ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&pv_done[x], (uint32_t)(done + steps - 1) & 1u));
                // (the queries' place is ours, with the gate's inputs in it)
                if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&z_full[x], (uint32_t)outs & 1u));
                if (!ok) break;
                tc::tc_fence_after();
                ++outs;
            }
            if (it.slot >= 0) {
                // a piece: the sums as they are, for the join (no sum where the second pass is to decide)
                const int64_t pr = (int64_t)it.slot * kSplitRows + x * kRows + row;
                if (live) plan.part_ml[pr] = make_float2(m, finite ? l : __int_as_float(0x7fffffff));
                if (steps > 0) {
                    if (lane == 0) tc::mbar_arrive(&q_empty[x]);
                    // [4 columns][row]: a warp's rows lie together in every store
                    float4* out = reinterpret_cast<float4*>(plan.part_o) + (pr - row) * (D / 4) + row;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        tc::tmem_ld16(to + c, o);
                        tc::tmem_wait_ld();
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                out[(c / 4 + e) * kRows] =
                                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                    }
                }
            } else if (steps == 0) {
                // no row of the tile sees a key, though the other tile's do
                if (live)
                    for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>((bf16*)a.o + at + c) = make_uint4(0, 0, 0, 0);
            } else {
                // O / sum, gated, as bf16 into shared memory, in the swizzled layout of the tile copies
                const bool empty = lim < 0;
                const float inv = empty ? 0.f : 1.0f / l;
                float bad = 0.f;                       // 0 * y: NaN once a y is not finite
                uint8_t* stage = q_smem + x * C::kTile + row * 128;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tc::tmem_ld32_raw(to + c, reinterpret_cast<uint32_t*>(o));
                    tc::tmem_wait_ld();
                    uint8_t* place = stage + (c >> 6) * C::kHalf;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint4* p = reinterpret_cast<uint4*>(place + (((((c & 32) >> 3) + e) ^ (row & 7)) << 4));
                        float y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            y[k] = empty ? 0.f : o[8 * e + k] * inv;
                            bad = fmaf(y[k], 0.f, bad);
                        }
                        if (a.z && !empty) {
                            const uint4 zz = *p;
                            const uint32_t w[4] = {zz.x, zz.y, zz.z, zz.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                y[2 * k] = gate_out_fast(y[2 * k], __uint_as_float(w[k] << 16));
                                y[2 * k + 1] = gate_out_fast(y[2 * k + 1], __uint_as_float(w[k] & 0xffff0000u));
                            }
                        }
                        *p = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                                        pack_bf16(y[6], y[7]));
                    }
                }
                if (bad != 0.f) finite = false;
                // out: a whole tile by a tile copy, what is left of a sequence row by row
                const bool whole = ntok == tokens;
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&staged[x]);
                if (whole) {
                    if (warp == 4 * x) {
                        ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&staged[x], (uint32_t)stages & 1u));
                        if (ok && lane == 0) {
                            for (int h = 0; h < C::kHalves; ++h)
                                tc::tma_store_3d(&to_map, q_smem + x * C::kTile + h * C::kHalf, h * 64, it.kvh * G,
                                                 it.q0 + it.tok + x * tokens);
                            tc::bulk_commit();
                            tc::bulk_wait_read<0>();
                        }
                        __syncwarp();
                    }
                } else {
                    ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&staged[x], (uint32_t)stages & 1u));
                    if (!ok) break;
                    constexpr int kLanes = D / 8;      // lanes to a row
                    const int sub = lane / kLanes, chunk = lane % kLanes;
#pragma unroll 1
                    for (int k = sub; k < 32; k += 32 / kLanes) {
                        const int rk = (warp & 3) * 32 + k, tk_ = rk / G;
                        if (tk_ >= ntok) break;
                        const uint4 v = *reinterpret_cast<const uint4*>(q_smem + x * C::kTile + (chunk >> 3) * C::kHalf + rk * 128 +
                                                                        (((chunk & 7) ^ (rk & 7)) << 4));
                        const int64_t to_row = ((int64_t)it.q0 + it.tok + x * tokens + tk_) * a.HQ + it.kvh * G + rk - tk_ * G;
                        *reinterpret_cast<uint4*>((bf16*)a.o + to_row * D + chunk * 8) = v;
                    }
                }
                ++stages;
                // The place is free for the next queries once every warp has said so: each has then seen
                // its phase of z_full (a warp that is still to look at one must not miss two), and read
                // its rows, or, the first warp, seen the tile copy read them.
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&q_empty[x]);
                if (__any_sync(0xffffffffu, !finite && live) && lane == 0)
                    list_redo(plan, it.n, it.kvh, (it.tok + x * tokens) * G + (warp & 3) * 32,
                              min(32, tokens * G - (warp & 3) * 32));
            }
            tc::tc_fence_before();       // the reads of O are over before the next item's weights are handed on
            t0 += 2 * it.total(tokens);
            done += steps;
            lasts += steps > 0 && steps == it.total(tokens);
        }
        if (lane == 0) tc::bulk_wait<0>();             // (the tile copies out are complete)
        if (!ok && lane == 0) s_timeout = 1;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
    if (tid == 0 && s_timeout) atomicMax(&g_attn_tc_error, GDN_DEVERR_TIMEOUT);
}

// Joins the pieces of a split plan.  Block (c - 1, y): rows 16 y .. 16 y + 15 of the (tile, head) that
// block c of the main kernel left to it; a thread one row and D / 64 chunks of four columns (the pieces
// lie as [4 columns][row]), kBatch pieces' loads in flight.  The outputs go through shared memory, so
// that gate inputs and outputs are read and written 16 bytes at a time along the rows.
constexpr int kJoinThreads = 256, kJoinRows = 16, kBatch = 4;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_rows_kernel(AttnArgs a, AttnPlan plan, int tokens) {
    constexpr int NC = D / 64, kStride = D + 4;
    __shared__ float s_y[kJoinRows * kStride];
    tc::grid_dependency_sync();
    const int c = blockIdx.x + 1;
    if (c >= plan.counts[3]) return;
    const int4 d = plan.desc[c];
    if (d.x < 0) return;
    const PlanTile t = plan.tiles[d.x];
    const int tid = threadIdx.x, G = a.HQ / a.HKV, h = d.y;
    const int r0 = blockIdx.y * kJoinRows, x = r0 / kRows, tr0 = r0 - x * kRows;
    const int tok0 = (t.index * 2 + x) * tokens;            // the half's first token
    const int rows = min(tokens, t.n_q - tok0) * G - tr0;   // the half's rows from r0 on
    if (rows <= 0) return;
    const int64_t to0 = ((int64_t)t.q0 + tok0) * a.HQ + (int64_t)h * G;
    bool finite = true;
    {
        const int row = tid % kJoinRows, chunk = tid / kJoinRows;
        float m = -INFINITY, l = 0.f;
        float4 o[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b0 = row < rows ? d.z : d.w + 1; b0 <= d.w; b0 += kBatch) {
            float2 ml[kBatch];
            float4 y[kBatch][NC];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int b = b0 + k;
                ml[k] = make_float2(-INFINITY, 0.f);
                if (b > d.w) continue;
                const int64_t half = ((int64_t)b * 2 + (b == d.z ? 1 : 0)) * kSplitRows + x * kRows;
                ml[k] = plan.part_ml[half + tr0 + row];
                const float4* p = reinterpret_cast<const float4*>(plan.part_o) + half * (D / 4) + tr0 + row;
#pragma unroll
                for (int i = 0; i < NC; ++i) y[k][i] = p[(chunk + i * 16) * kRows];
            }
            float mn = m;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ml[k].x);
            const float base = mn == -INFINITY ? 0.f : mn;
            const float g = exp2_sfu(m - base);
            m = mn;
            l *= g;
#pragma unroll
            for (int i = 0; i < NC; ++i) o[i] = make_float4(o[i].x * g, o[i].y * g, o[i].z * g, o[i].w * g);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                // (a piece in which the row sees no key has no sums, whatever lies there)
                if (ml[k].x == -INFINITY && ml[k].y == 0.f) continue;
                const float f = exp2_sfu(ml[k].x - base);
                l = fmaf(f, ml[k].y, l);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    o[i].x = fmaf(f, y[k][i].x, o[i].x);
                    o[i].y = fmaf(f, y[k][i].y, o[i].y);
                    o[i].z = fmaf(f, y[k][i].z, o[i].z);
                    o[i].w = fmaf(f, y[k][i].w, o[i].w);
                }
            }
        }
        if (row < rows) {
            const bool empty = t.n_kv - t.n_q + tok0 + (tr0 + row) / G < 0;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const float4 v = empty ? make_float4(0.f, 0.f, 0.f, 0.f)
                                       : make_float4(o[i].x / l, o[i].y / l, o[i].z / l, o[i].w / l);
                // 0 * v: NaN once a v is not finite
                const float bad = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, v.w * 0.f)));
                finite = finite && bad == 0.f;
                *reinterpret_cast<float4*>(s_y + row * kStride + (chunk + i * 16) * 4) = v;
            }
        }
    }
    const bool redo = __syncthreads_or(!finite);
    for (int u = tid; u < kJoinRows * (D / 8); u += kJoinThreads) {
        const int row = u / (D / 8), col = u % (D / 8) * 8, tr = tr0 + row;
        if (row >= rows) break;
        const int64_t to = (to0 + (int64_t)(tr / G) * a.HQ + tr % G) * D + col;
        const float* y = s_y + row * kStride + col;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = y[e];
        if (a.z && t.n_kv - t.n_q + tok0 + tr / G >= 0) {
            const uint4 zz = *reinterpret_cast<const uint4*>((const bf16*)a.z + to);
            const uint32_t w[4] = {zz.x, zz.y, zz.z, zz.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = gate_out_fast(v[2 * e], __uint_as_float(w[e] << 16));
                v[2 * e + 1] = gate_out_fast(v[2 * e + 1], __uint_as_float(w[e] & 0xffff0000u));
            }
        }
        *reinterpret_cast<uint4*>((bf16*)a.o + to) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
    // (rows are listed as the (token, head) rows of the sequence)
    if (redo && tid == 0) list_redo(plan, t.n, h, tok0 * G + tr0, min(kJoinRows, tokens * G - tr0));
}

// The workspace: the plan's, then what the kernel for short pieces wants.
constexpr int kRedoPerHead = kSplitRows / kJoinRows;      // records of a (tile, key-value head), at most: the join's
AttnPlan plan_of(void* ws, int64_t n_tokens, int n_seqs, int HQ, int HKV, int D) {
    return attn_plan(ws, n_tokens, n_seqs, kRedoPerHead * HKV, 1, 2 * (kRows / (HQ / HKV)), HKV, D);
}
size_t short_at(const AttnPlan& plan) { return (plan.bytes + 255) / 256 * 256; }

template <int D>
cudaError_t launch_tiles(const AttnArgs& a, const AttnPlan& plan, int blocks, cudaStream_t s) {
    using C = Cfg<D>;
    const int G = a.HQ / a.HKV, tokens = kRows / G;
    cudaError_t e;
    CUtensorMap tq, tk, tv, tz, to;
    const int page = 1 << a.kv.page_shift;
    const int box_rows = a.kv.table && page < kKeys ? page : kKeys;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.HQ, (cuuint64_t)a.n_tokens};
        const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.HQ * D * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tokens};
        if (!make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_map(&tz, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.z ? a.z : a.q, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_map(&to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.o, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    const int64_t kv_rows = a.kv.table ? (int64_t)a.kv.n_pages << a.kv.page_shift : a.n_tokens;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.HKV, (cuuint64_t)kv_rows};
    const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.HKV * D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
    if (!make_map(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv.k, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv.v, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    e = allow_smem((const void*)attn_prefill_kernel<D>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    // (a plan that may split is for the whole grid, however few its tiles)
    const int64_t most = (int64_t)plan.max_tiles * a.HKV;
    const int grid = plan.can_split || most > blocks ? blocks : (int)most;
    e = launch_pdl(attn_prefill_kernel<D>, dim3((unsigned)grid), dim3(kThreads), C::kSmem, s, tq, tk,
                   tv, tz, to, a, plan, tokens, box_rows);
    if (e != cudaSuccess) return e;
    count_launch();
    if (plan.can_split && grid > 1) {
        e = launch_pdl(attn_join_rows_kernel<D>, dim3((unsigned)(grid - 1), kSplitRows / kJoinRows), dim3(kJoinThreads), 0, s, a,
                       plan, tokens);
        if (e != cudaSuccess) return e;
        count_launch();
    }
    return cudaSuccess;
}

}  // namespace

bool attn_tc_supported(int HQ, int HKV) { return HQ / HKV <= kRows; }

size_t attn_tc_bytes(int64_t n_tokens, int n_seqs, int HQ, int HKV, int D) {
    const AttnPlan plan = plan_of(nullptr, n_tokens, n_seqs, HQ, HKV, D);
    // the list of rows to do again is counted in 32 bits (many millions of sequences pass that)
    if ((int64_t)plan.max_tiles * kRedoPerHead * HKV > INT32_MAX) return 0;
    return short_at(plan) + attn_decode_bytes(D);
}

cudaError_t launch_attn_tc(const AttnArgs& args, cudaStream_t s) {
    AttnArgs a = args;
    const int G = a.HQ / a.HKV;
    const AttnPlan plan = plan_of(a.ws, a.n_tokens, a.n_seqs, a.HQ, a.HKV, a.D);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int blocks = sms < kSplitGrid ? sms : kSplitGrid;
    // Pieces of a few rows (drafts, single tokens) leave most of a tile's rows idle and pay its chain of
    // products and softmax per step, so they are streamed instead.  Lengths are on the device: here it
    // is decided by the mean, since two passes one after the other lose where few pieces are short.
    // Streamed against tiles at a mean of 16 rows: 80 against 102 us (64 x 4 tokens, 32 heads over 8, past
    // 1000), 65 / 69 (8 x 4, 16 over 4, 16000); 4: 67 / 83 (64 x 1, 2000); 32: 42 / 35 (16 x 8); 35, one
    // piece of 512 and 63 tokens: 100 / 96.
    if (a.kv.table && a.n_tokens * G <= (int64_t)kShortRows * a.n_seqs) a.short_rows = kShortRows;
    const bool all_short = a.short_rows > 0 && a.n_tokens * G <= kShortRows;
    e = launch_attn_plan(a, plan, 1, 2 * (kRows / G), blocks, s);
    if (e == cudaSuccess && !all_short)
        e = a.D == 128 ? launch_tiles<128>(a, plan, blocks, s) : launch_tiles<64>(a, plan, blocks, s);
    if (e == cudaSuccess && a.short_rows > 0)
        e = launch_attn_short(a, plan, static_cast<uint8_t*>(a.ws) + short_at(plan), s);
    return e == cudaSuccess ? launch_attn_redo(a, plan, s) : e;
}

cudaError_t read_attn_tc_error(int32_t* out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_attn_tc_error, sizeof(int32_t));
    if (e == cudaSuccess && *out != 0) {
        const int32_t zero = 0;
        e = cudaMemcpyToSymbol(g_attn_tc_error, &zero, sizeof(int32_t));
    }
    return e;
}

}  // namespace gdn
