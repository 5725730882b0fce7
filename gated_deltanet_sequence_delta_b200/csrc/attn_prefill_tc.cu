// attn_prefill_tc.cu -- causal grouped attention of prompts on the tensor cores (bf16).
//
//   S = scale Q K^T,  P = e^{S - m} (0 where a row does not see a key),  O = P V / rowsum(P)
//
// in one pass over the keys with a running reference m per row.  FLOPs: 4 D per (row, key) pair,
// 2 D x 2 products; bound by the tensor cores and, at D = 64, by the exponentials: an SM takes
// 16 of them a clock in its special-function units, so the 128 x 128 weights of a step cost 1024
// clocks there against 1024 (D = 128) or 512 (D = 64) of the two products.  A share of them is
// therefore formed on the FMA pipes (exp2_poly).
//
// Rows.  A tile is 128 rows, the (token, query head of the group) pairs of one key-value head:
// 128 / G tokens by G heads, so that the group shares every key and value that is staged and
// the diagonal's waste shrinks with G (rows left over where G does not divide 128 are idle).  A
// block takes two consecutive tiles, A and B, against the same keys: while the softmax of one
// runs, the tensor cores work for the other.  Blocks are persistent, so that an item's first
// loads and scores run under the last item's outputs.
//
// Roles (12 warps, one block per SM; the last only completes a warpgroup):
//   warps 0-3, 4-7   softmax of tile A, of tile B: a thread owns a row (TMEM lane), takes its 128
//                    scores into registers, forms the weights, writes them as bf16
//   warps 8, 9       issue the MMAs of tile A, of tile B: per step  S = Q K',  O += P V  (K' the
//                    next step's keys); two warps, so that neither tile's products wait behind
//                    the other's softmax
//   warp 10          TMA: queries once, then keys and values through a ring
// TMEM, 512 columns: S 128, P_A and P_B 64 each, O_A and O_B D each.  A tile's scores of the next
// step are formed while its softmax works on the last ones, so that the products stay off that
// chain; at D = 128 this leaves room for one S, which the tiles use in turn (it is free again
// once its softmax warps have read it), at D = 64 for one each.
//
// The reference m moves only when a row's maximum has grown by more than 2^8 since it was set:
// weights then stay below 2^8, sums and products in fp32 lose nothing, and the accumulated O has
// to be rescaled in tensor memory only in a row's first steps.  The weights are rounded to bf16
// for the product (half a step, 2^-8 relative, each); their sum is taken before the rounding.
//
// Masked weights are exact zeros, but 0 * v is not 0 where v is infinite or NaN.  Values past
// the last key that any row of the block sees are cleared in shared memory; a value inside the
// diagonal that is not finite shows in the outputs, whose tile is then put on a list that the
// CUDA-core kernel, which leaves masked places out of its sums, does again.
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
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;            // growth of the maximum (log2) that moves the reference

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

// 2^x for two floats, |x| < 126 or x < 0 (below 2^-126 it stays there): x = n + f, n the nearest
// integer by the magic-number addition, 2^f on [-1/2, 1/2] by the cubic of least relative error
// (7.5e-5, found by the Remez exchange), n added to the exponent field.
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
__device__ __forceinline__ void exp2_poly(float& a, float& b) {
    const uint64_t x = pack2(fmaxf(a, -126.0f), fmaxf(b, -126.0f));
    const uint64_t magic = pack2(12582912.0f, 12582912.0f);
    const uint64_t t = add2(x, magic);
    const uint64_t n = add2(t, pack2(-12582912.0f, -12582912.0f));
    const uint64_t f = fma2(n, pack2(-1.0f, -1.0f), x);
    uint64_t p = fma2(f, pack2(0.05517166852951050f, 0.05517166852951050f),
                      pack2(0.2426111251115799f, 0.2426111251115799f));
    p = fma2(p, f, pack2(0.6932609677314758f, 0.6932609677314758f));
    p = fma2(p, f, pack2(0.9999280571937561f, 0.9999280571937561f));
    float pa, pb, ta, tb;
    unpack2(p, pa, pb);
    unpack2(t, ta, tb);
    a = __int_as_float(__float_as_int(pa) + (__float_as_int(ta) << 23));
    b = __int_as_float(__float_as_int(pb) + (__float_as_int(tb) << 23));
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
// their sum.  `free` is called before the first write.  MASKED: keys past `last` weigh exactly 0,
// and all the others go through the special-function units (the cubic does not reach 0).
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
            } else if ((j & 7) == 6) {
                exp2_poly(e0, e1);
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

// One item of a block's work: tiles A and B of a (sequence, tile pair, key-value head).
struct Item {
    int n, kvh, q0, n_q, n_kv, past;
    int tok;                   // first token of A; B follows `tokens` later
    int tokens;
    // of tile x: tokens it has (0: no tile), keys its last row sees, steps of 128 keys
    __device__ __forceinline__ int ntok(int x) const { return max(min(tokens, n_q - tok - x * tokens), 0); }
    __device__ __forceinline__ int end(int x) const { return ntok(x) > 0 ? max(past + tok + x * tokens + ntok(x), 0) : 0; }
    __device__ __forceinline__ int steps(int x) const { return (end(x) + kKeys - 1) / kKeys; }
    __device__ __forceinline__ int total() const { return max(steps(0), steps(1)); }
};
// The r-th item of this block.  The list runs from long to short; blocks take it forwards and
// backwards in turn, which evens out their sums.
__device__ __forceinline__ bool item_at(const AttnArgs& a, const AttnPlan& plan, int count, int tokens, int r, Item& it) {
    const int64_t i = (int64_t)r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (i >= count) return false;
    const int2 pt = plan.tiles[i / a.HKV];
    const SeqRows sq = seq_rows(a, pt.x);
    it.n = pt.x;
    it.kvh = (int)(i % a.HKV);
    it.q0 = sq.q0;
    it.n_q = sq.n_q;
    it.n_kv = sq.n_kv;
    it.past = sq.n_kv - sq.n_q;
    it.tok = pt.y * 2 * tokens;
    it.tokens = tokens;
    return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(const __grid_constant__ CUtensorMap tq,
                                                                   const __grid_constant__ CUtensorMap tk,
                                                                   const __grid_constant__ CUtensorMap tv, AttnArgs a,
                                                                   AttnPlan plan, int tokens, int box_rows) {
    using C = Cfg<D>;
    constexpr int S = C::kRing;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t q_full, q_empty, kv_full[S], kv_empty[S], s_full[2], s_read[2], p_full[2], pv_done[2],
        drain[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_timeout;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* q_smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* ring = q_smem + 2 * C::kTile;
    const int G = a.HQ / a.HKV;

    if (tid == 0) {
        tc::mbar_init(&q_full, 1);
        tc::mbar_init(&q_empty, 2);
        for (int i = 0; i < S; ++i) {
            tc::mbar_init(&kv_full[i], 1);
            tc::mbar_init(&kv_empty[i], 2);
        }
        for (int x = 0; x < 2; ++x) {
            tc::mbar_init(&s_full[x], 1);
            tc::mbar_init(&s_read[x], 4);
            tc::mbar_init(&p_full[x], 4);
            tc::mbar_init(&pv_done[x], 1);
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
    const int count = plan.counts[0] * a.HKV;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 10) {
            // ---- loads ------------------------------------------------------------------
            bool ok = true;
            const int boxes = kKeys / box_rows;
            const int lg = lane / C::kHalves, lh = lane % C::kHalves;  // this lane's box, its column block
            const int none = (int)((int64_t)a.kv.n_pages << a.kv.page_shift);
            int t = 0, items = 0;
            Item it;
            for (int r = 0; ok && item_at(a, plan, count, tokens, r, it); ++r) {
                const int total = it.total();
                for (int u = 0; u < 2 * total; ++u, ++t) {             // K_0, (Q), K_1, V_0, K_2, V_1, ..., V_last
                    const bool is_v = u + 1 == 2 * total || (u > 0 && (u & 1) == 0);
                    const int step = u + 1 == 2 * total ? total - 1 : is_v ? (u >> 1) - 1 : (u + 1) >> 1;
                    if (u == 1) {
                        if (items > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(&q_empty, (uint32_t)(items - 1) & 1u));
                        if (!ok) break;
                        if (lane == 0) {
                            const int tiles = it.ntok(1) > 0 ? 2 : 1;
                            tc::mbar_expect_tx(&q_full, (uint32_t)(tiles * C::kHalves * tokens * G * 128));
                            for (int x = 0; x < tiles; ++x)
                                for (int h = 0; h < C::kHalves; ++h)
                                    tc::tma_load_3d(q_smem + x * C::kTile + h * C::kHalf, &tq, &q_full, h * 64, it.kvh * G,
                                                    it.q0 + it.tok + x * tokens);
                        }
                        __syncwarp();
                        ++items;
                    }
                    const int s = t % S;
                    const int pos = step * kKeys + lg * box_rows;
                    int row = it.q0 + pos;
                    if (a.kv.table && lg < boxes) {
                        row = none;                                    // past the cache: zero fill
                        if (pos < it.n_kv) {
                            const int64_t c = cache_row(a.kv.table + (int64_t)it.n * a.kv.max_pages, pos, a.kv.page_shift,
                                                        a.kv.n_pages);
                            if (c >= 0)
                                row = (int)c;
                            else
                                atomicMax(&g_attn_tc_error, GDN_DEVERR_PAGE);
                        }
                    }
                    if (t >= S) ok = __all_sync(0xffffffffu, tc::mbar_wait(&kv_empty[s], (uint32_t)((t / S) & 1) ^ 1u));
                    if (!ok) break;
                    if (lane == 0) tc::mbar_expect_tx(&kv_full[s], C::kTile);
                    __syncwarp();
                    if (lg < boxes)
                        tc::tma_load_3d(ring + s * C::kTile + lh * C::kHalf + lg * box_rows * 128, is_v ? &tv : &tk,
                                        &kv_full[s], lh * 64, it.kvh, row);
                }
            }
            if (!ok) {       // an expired wait: give the copies under way time to land
                if (lane == 0) s_timeout = 1;
                for (int i = 0; i < S; ++i) tc::mbar_wait(&kv_full[i], (uint32_t)(((t - 1 - i) / S) & 1), 1000000);
            }
        } else if (warp < 10) {
            // ---- products of tile x ---------------------------------------------------------
            // (the whole warp walks the loop, one elected lane issues)
            const int x = warp - 8;
            const uint32_t neg = a.scale < 0.f ? 1u << 13 : 0u;        // -Q: scores of a negative scale
            const uint32_t id_s = tc::idesc_bf16(128, kKeys, 0, 0) | neg, id_o = tc::idesc_bf16(128, D, 0, 1);
            const uint64_t qd = tc::desc_sw128(tc::smem_u32(q_smem + x * C::kTile), 0, 1024);
            const uint64_t kd = tc::desc_sw128(tc::smem_u32(ring), 0, 1024), vd = tc::desc_sw128(tc::smem_u32(ring), C::kHalf, 1024);
            bool ok = true;
            int t0 = 0, items = 0, mine = 0, others = 0;               // ring tiles, items and steps before this item
            int last = -1;                                             // the tile that used S last
            auto wait = [&](uint64_t* bar, int phase) {
                if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, (uint32_t)phase & 1u));
            };
            auto wait_kv = [&](int t) { wait(&kv_full[t % S], t / S); };
            Item it;
            for (int r = 0; ok && item_at(a, plan, count, tokens, r, it); ++r) {
                const int steps = it.steps(x), other = it.steps(x ^ 1), total = it.total();
                if (total == 0) continue;
                wait(&q_full, items);
                ++items;
                for (int i = -1; i < total && ok; ++i) {               // S(i + 1), then O += P(i) V(i)
                    if (i + 1 < total) {
                        const int t = i < 0 ? t0 : t0 + 2 * i + 1;     // ring tile of K(i + 1)
                        wait_kv(t);
                        if (i + 1 < steps) {
                            // S is free once its last user has read it: the other tile's turn
                            // between ours, or whichever came last
                            if (!C::kOneS) {
                                if (mine + i >= 0) wait(&s_read[x], mine + i);
                            } else if (x == 0 ? i >= 0 && i < other : i + 1 < other) {
                                wait(&s_read[x ^ 1], others + i + x);
                            } else if (i >= 0) {
                                wait(&s_read[x], mine + i);
                            } else if (last >= 0) {
                                wait(&s_read[last], (last == x ? mine : others) - 1);
                            }
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
                                if (i + 2 == steps) tc::mma_commit(&q_empty);
                            }
                        } else if (ok && lane == 0) {
                            tc::mbar_arrive(&kv_empty[t % S]);         // a tile of keys that only the other tile takes
                            if (i < 0) tc::mbar_arrive(&q_empty);
                        }
                        __syncwarp();
                    }
                    if (i < 0) continue;
                    const int t = t0 + (i + 1 < total ? 2 * i + 2 : 2 * i + 1);       // ring tile of V(i)
                    wait_kv(t);
                    if (i < steps) {
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
                    } else if (ok && lane == 0) {
                        tc::mbar_arrive(&kv_empty[t % S]);
                    }
                    __syncwarp();
                }
                t0 += 2 * total;
                mine += steps;
                others += other;
                last = it.steps(1) == total ? 1 : 0;
            }
            // every arrival of the commits above has landed before the block leaves
            if (tc::elect_one()) tc::mma_commit(&drain[x]);
            __syncwarp();
            if (!tc::mbar_wait(&drain[x], 0) || !ok) s_timeout = 1;
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
        int t0 = 0, done = 0;                                          // ring tiles and steps before this item
        Item it;
        for (int r = 0; ok && item_at(a, plan, count, tokens, r, it); ++r) {
            const int steps = it.steps(x), total = it.total();
            // last key this row sees (idle rows: no mask; nothing of them is kept)
            const int lim = tok < it.ntok(x) ? it.past + it.tok + x * tokens + tok : INT32_MAX;
            // the tile that clears the values past the item's last key: the first such key
            const int clear_from = x == (it.steps(0) == total ? 0 : 1) ? max(it.end(0), it.end(1)) : INT32_MAX;
            float m = -INFINITY, l = 0.f;
            bool finite = true;
            for (int i = 0; i < steps; ++i) {
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&s_full[x], (uint32_t)(done + i) & 1u));
                if (!ok) break;
                tc::tc_fence_after();
                float s[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) tc::tmem_ld32_raw(ts + c, reinterpret_cast<uint32_t*>(s) + c);
                tc::tmem_wait_ld();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&s_read[x]);
                const int j0 = i * kKeys;
                const bool masked = __any_sync(0xffffffffu, j0 + kKeys - 1 > lim);
                if (masked) {
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (j0 + j > lim) s[j] = -INFINITY;
                }
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
                        ok = __all_sync(0xffffffffu, tc::mbar_wait(&pv_done[x], (uint32_t)(done + i - 1) & 1u));
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
                if (clear_from - j0 < kKeys) {
                    // values that no row of the block sees may be anything: clear them
                    const int t = t0 + 2 * total - 1, slot = t % S;           // the item's last values
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&kv_full[slot], (uint32_t)((t / S) & 1)));
                    if (!ok) break;
                    uint8_t* v = ring + slot * C::kTile;
                    const int first = clear_from - j0;
                    for (int e = row; e < (kKeys - first) * 8 * C::kHalves; e += 128) {
                        const int vr = first + e / (8 * C::kHalves), c = e % (8 * C::kHalves);
                        *reinterpret_cast<uint4*>(v + (c >> 3) * C::kHalf + vr * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_async_smem();
                }
                const float base = m == -INFINITY ? 0.f : m;
                auto free = [&] {                        // the last step's product has read P
                    if (i > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(&pv_done[x], (uint32_t)(done + i - 1) & 1u));
                    tc::tc_fence_after();
                };
                if (masked)
                    l += weights<true>(s, sc, base, lim - j0, tp, free);
                else
                    l += weights<false>(s, sc, base, 0, tp, free);
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (!ok) break;
                if (lane == 0) tc::mbar_arrive(&p_full[x]);
            }
            if (!ok) break;
            if (steps > 0) {
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&pv_done[x], (uint32_t)(done + steps - 1) & 1u));
                if (!ok) break;
                tc::tc_fence_after();
            }
            item_at(a, plan, count, tokens, r, it);       // (again: not kept in registers over the loop)
            const bool live = tok < it.ntok(x), empty = lim < 0;
            const float inv = empty ? 0.f : 1.0f / l;
            const int64_t at = (((int64_t)it.q0 + it.tok + x * tokens + tok) * a.HQ + it.kvh * G + g) * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                if (steps > 0) {
                    tc::tmem_ld32_raw(to + c, reinterpret_cast<uint32_t*>(o));
                    tc::tmem_wait_ld();
                }
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        o[e] = empty ? 0.f : o[e] * inv;
                        finite = finite && fabsf(o[e]) <= 3.4028235e38f;
                    }
                    if (a.z && !empty) {
                        const uint4* z = reinterpret_cast<const uint4*>((const bf16*)a.z + at + c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 zz = z[e];
                            const uint32_t w[4] = {zz.x, zz.y, zz.z, zz.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                o[e * 8 + 2 * k] = gate_out(o[e * 8 + 2 * k], __uint_as_float(w[k] << 16));
                                o[e * 8 + 2 * k + 1] = gate_out(o[e * 8 + 2 * k + 1], __uint_as_float(w[k] & 0xffff0000u));
                            }
                        }
                    }
                    uint4* out = reinterpret_cast<uint4*>((bf16*)a.o + at + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        out[e] = make_uint4(pack_bf16(o[e * 8], o[e * 8 + 1]), pack_bf16(o[e * 8 + 2], o[e * 8 + 3]),
                                            pack_bf16(o[e * 8 + 4], o[e * 8 + 5]), pack_bf16(o[e * 8 + 6], o[e * 8 + 7]));
                }
            }
            if (__any_sync(0xffffffffu, !finite && live) && lane == 0) {
                // (rows of a bad table may be listed twice: never past the list's end)
                const int k = atomicAdd(&plan.counts[1], 1);
                if (k < plan.max_redo)
                    plan.redo[k] = make_int4(it.n, it.kvh, (it.tok + x * tokens) * G + (warp & 3) * 32,
                                             min(32, tokens * G - (warp & 3) * 32));
            }
            tc::tc_fence_before();       // the reads of O are over before the next item's weights are handed on
            t0 += 2 * it.total();
            done += steps;
        }
        if (!ok && lane == 0) s_timeout = 1;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
    if (tid == 0 && s_timeout) atomicMax(&g_attn_tc_error, GDN_DEVERR_TIMEOUT);
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    using C = Cfg<D>;
    const int G = a.HQ / a.HKV, tokens = kRows / G;
    const AttnPlan plan = attn_plan(a.ws, a.n_tokens, a.n_seqs, 8 * a.HKV, 1, 2 * tokens);
    cudaError_t e = launch_attn_plan(a, plan, 1, 2 * tokens, s);
    if (e != cudaSuccess) return e;
    CUtensorMap tq, tk, tv;
    const int page = 1 << a.kv.page_shift;
    const int box_rows = a.kv.table && page < kKeys ? page : kKeys;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.HQ, (cuuint64_t)a.n_tokens};
        const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.HQ * D * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tokens};
        if (!make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    const int64_t kv_rows = a.kv.table ? (int64_t)a.kv.n_pages << a.kv.page_shift : a.n_tokens;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.HKV, (cuuint64_t)kv_rows};
    const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.HKV * D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
    if (!make_map(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv.k, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv.v, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    e = cudaFuncSetAttribute(attn_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)plan.max_tiles * a.HKV;
    e = launch_pdl(attn_prefill_kernel<D>, dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads), C::kSmem, s, tq, tk,
                   tv, a, plan, tokens, box_rows);
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_attn_redo(a, plan, s);
}

}  // namespace

bool attn_tc_supported(int HQ, int HKV) { return HQ / HKV <= kRows; }

size_t attn_tc_bytes(int64_t n_tokens, int n_seqs, int HQ, int HKV) {
    const AttnPlan p = attn_plan(nullptr, n_tokens, n_seqs, 8 * HKV, 1, 2 * (kRows / (HQ / HKV)));
    return p.bytes;
}

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s) { return a.D == 128 ? launch<128>(a, s) : launch<64>(a, s); }

cudaError_t read_attn_tc_error(int32_t* out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_attn_tc_error, sizeof(int32_t));
    if (e == cudaSuccess && *out != 0) {
        const int32_t zero = 0;
        e = cudaMemcpyToSymbol(g_attn_tc_error, &zero, sizeof(int32_t));
    }
    return e;
}

}  // namespace gdn
