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
// runs, the tensor cores work for the other.
//
// Roles (12 warps, one block per SM; warps 10 and 11 only complete a warpgroup):
//   warps 0-3, 4-7   softmax of tile A, of tile B: a thread owns a row (TMEM lane), reads its 128
//                    scores, forms the weights, writes them as bf16 over the scores
//   warp 8           issues the MMAs: per step  O_A += P_A V,  S_A = Q_A K',  O_B += P_B V,
//                    S_B = Q_B K'  (K' the next keys)
//   warp 9           TMA: queries once, then keys and values through a ring
// TMEM: S_A, S_B (128 columns each, the weights in the first 64), O_A, O_B (D columns each).
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

// The block's work: tiles A and B of one (sequence, tile pair, key-value head).
struct Item {
    SeqRows sq;
    int n, kvh, past;
    int tok[2], ntok[2];       // first token of each tile, tokens in it (0: no tile)
    int steps[2];              // key steps of each tile
    int total;
};
__device__ __forceinline__ Item item_of(const AttnArgs& a, int n, int pair, int kvh, int tokens) {
    Item it;
    it.n = n;
    it.kvh = kvh;
    it.sq = seq_rows(a, n);
    it.past = it.sq.n_kv - it.sq.n_q;
    it.total = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        it.tok[x] = (pair * 2 + x) * tokens;
        it.ntok[x] = max(min(tokens, it.sq.n_q - it.tok[x]), 0);
        const int end = it.ntok[x] > 0 ? max(it.past + it.tok[x] + it.ntok[x], 0) : 0;    // keys its last row sees
        it.steps[x] = (end + kKeys - 1) / kKeys;
        it.total = max(it.total, it.steps[x]);
    }
    return it;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(const __grid_constant__ CUtensorMap tq,
                                                                   const __grid_constant__ CUtensorMap tk,
                                                                   const __grid_constant__ CUtensorMap tv, AttnArgs a,
                                                                   AttnPlan plan, int tokens, int box_rows) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t q_full, kv_full[C::kRing], kv_empty[C::kRing], s_full[2], p_full[2], o_full[2],
        drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_redo, s_timeout;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((int)(blockIdx.x / a.HKV) >= plan.counts[0]) return;
    uint8_t* q_smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* ring = q_smem + 2 * C::kTile;
    const int G = a.HQ / a.HKV;
    const int2 pt = plan.tiles[blockIdx.x / a.HKV];
    const Item it = item_of(a, pt.x, pt.y, blockIdx.x % a.HKV, tokens);

    if (tid == 0) {
        tc::mbar_init(&q_full, 1);
        for (int i = 0; i < C::kRing; ++i) {
            tc::mbar_init(&kv_full[i], 1);
            tc::mbar_init(&kv_empty[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            tc::mbar_init(&s_full[x], 1);
            tc::mbar_init(&p_full[x], 4);
            tc::mbar_init(&o_full[x], 1);
        }
        tc::mbar_init(&drain, 1);
        tc::fence_mbar_init();
        s_redo = 0;
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

    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 9) {
        // ---- loads --------------------------------------------------------------------
        bool ok = true;
        if (lane == 0 && it.total > 0) {
            tc::mbar_expect_tx(&q_full, (uint32_t)((it.ntok[1] > 0 ? 2 : 1) * C::kHalves * tokens * G * 128));
            for (int x = 0; x < 2; ++x)
                if (it.ntok[x] > 0)
                    for (int h = 0; h < C::kHalves; ++h)
                        tc::tma_load_3d(q_smem + x * C::kTile + h * C::kHalf, &tq, &q_full, h * 64, it.kvh * G,
                                        it.sq.q0 + it.tok[x]);
        }
        const int boxes = kKeys / box_rows;
        const int lg = lane / C::kHalves, lh = lane % C::kHalves;      // this lane's box, its column block
        const int none = a.kv.table ? (int)((int64_t)a.kv.n_pages << a.kv.page_shift) : 0;
        for (int t = 0; t < 2 * it.total; ++t) {                        // K_0, V_0, K_1, V_1, ...
            const int s = t % C::kRing;
            if (t >= C::kRing) ok = __all_sync(0xffffffffu, tc::mbar_wait(&kv_empty[s], (uint32_t)((t / C::kRing) & 1) ^ 1u));
            if (!ok) break;
            const int pos = (t >> 1) * kKeys + lg * box_rows;
            uint8_t* dst = ring + s * C::kTile + lh * C::kHalf + lg * box_rows * 128;
            int row = it.sq.q0 + pos;
            if (a.kv.table && lg < boxes) {
                row = none;                                             // past the cache: zero fill
                if (pos < it.sq.n_kv) {
                    const int64_t r = cache_row(a.kv.table + (int64_t)it.n * a.kv.max_pages, pos, a.kv.page_shift,
                                                a.kv.n_pages);
                    if (r >= 0)
                        row = (int)r;
                    else
                        atomicMax(&g_attn_tc_error, GDN_DEVERR_PAGE);
                }
            }
            if (lane == 0) tc::mbar_expect_tx(&kv_full[s], C::kTile);
            __syncwarp();
            if (lg < boxes) tc::tma_load_3d(dst, (t & 1) ? &tv : &tk, &kv_full[s], lh * 64, it.kvh, row);
        }
        if (!ok) {
            if (lane == 0) s_timeout = 1;
            for (int i = 0; i < C::kRing; ++i) tc::mbar_wait(&kv_full[i], 0, 1000000);
        }
    } else if (warp == 8) {
        // ---- products -----------------------------------------------------------------
        if (lane == 0 && it.total > 0) {
            const uint32_t neg = a.scale < 0.f ? 1u << 13 : 0u;         // -Q: scores of a negative scale
            const uint32_t id_s = tc::idesc_bf16(128, kKeys, 0, 0) | neg, id_o = tc::idesc_bf16(128, D, 0, 1);
            bool ok = tc::mbar_wait(&q_full, 0);
            auto scores = [&](int x, int t) {                           // S_x = Q_x K^T, keys in ring tile t
                const uint32_t qa = tc::smem_u32(q_smem + x * C::kTile);
                const uint32_t kb = tc::smem_u32(ring + (t % C::kRing) * C::kTile);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k >> 2) * C::kHalf + (k & 3) * 32;
                    tc::mma_bf16(tmem + x * 128, tc::desc_sw128(qa + off, 0, 1024), tc::desc_sw128(kb + off, 0, 1024),
                                 id_s, k > 0);
                }
                tc::mma_commit(&s_full[x]);
            };
            auto outputs = [&](int x, int t, bool acc) {                // O_x += P_x V, values in ring tile t
                const uint32_t vb = tc::smem_u32(ring + (t % C::kRing) * C::kTile);
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    tc::mma_bf16_ts(tmem + 256 + x * D, tmem + x * 128 + k * 8,
                                    tc::desc_sw128(vb + k * 2048, C::kHalf, 1024), id_o, acc || k > 0);
            };
            auto wait_kv = [&](int t) {
                if (ok) ok = tc::mbar_wait(&kv_full[t % C::kRing], (uint32_t)((t / C::kRing) & 1));
                tc::tc_fence_after();
            };
            wait_kv(0);
            for (int x = 0; x < 2 && ok; ++x)
                if (it.steps[x] > 0) scores(x, 0);
            if (ok && C::kRing < 2 * it.total) tc::mma_commit(&kv_empty[0]);
            for (int i = 0; i < it.total && ok; ++i) {
                wait_kv(2 * i + 1);
                bool have_k = false;
                for (int x = 0; x < 2 && ok; ++x) {
                    if (i >= it.steps[x]) continue;
                    ok = tc::mbar_wait_spin(&p_full[x], (uint32_t)(i & 1));
                    if (!ok) break;
                    tc::tc_fence_after();
                    outputs(x, 2 * i + 1, i > 0);
                    if (i + 1 == it.steps[x]) tc::mma_commit(&o_full[x]);
                    if (i + 1 < it.steps[x]) {
                        if (!have_k) wait_kv(2 * i + 2);
                        have_k = true;
                        if (!ok) break;
                        scores(x, 2 * i + 2);
                    }
                }
                // (no arrival that nobody waits for: it could land after the block has left)
                for (int t = 2 * i + 1; ok && t <= 2 * i + (have_k ? 2 : 1); ++t)
                    if (t + C::kRing < 2 * it.total) tc::mma_commit(&kv_empty[t % C::kRing]);
            }
            if (!ok) {
                s_timeout = 1;
                tc::mma_commit(&drain);
                tc::mbar_wait(&drain, 0);
            }
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---- softmax: thread = row -------------------------------------------------------
        const int x = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const int steps = it.steps[x];
        const int tok = row / G;
        const bool live = tok < it.ntok[x];
        // last key this row sees (idle rows: no mask; nothing of them is kept)
        const int lim = live ? it.past + it.tok[x] + tok : INT32_MAX;
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;         // TMEM lane 32 (warp % 4)
        const uint32_t ts = tmem + lane_base + x * 128, to = tmem + lane_base + 256 + x * D;
        const float sc = fabsf(a.scale) * kLog2e;
        // the tile that clears the values past the item's last key
        const bool clears = x == (it.steps[0] == it.total ? 0 : 1);
        const int kv_end = max(it.past + (it.ntok[1] > 0 ? it.tok[1] + it.ntok[1] : it.tok[0] + it.ntok[0]), 0);
        float m = -INFINITY, l = 0.f;
        bool ok = true, finite = true;
        for (int i = 0; i < steps; ++i) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&s_full[x], (uint32_t)(i & 1)));
            if (!ok) break;
            tc::tc_fence_after();
            float s[128];
#pragma unroll
            for (int c = 0; c < 128; c += 32) tc::tmem_ld32_raw(ts + c, reinterpret_cast<uint32_t*>(s) + c);
            tc::tmem_wait_ld();
            const int j0 = i * kKeys;
            const bool masked = __any_sync(0xffffffffu, j0 + kKeys - 1 > lim);
            if (masked) {
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    if (j0 + j > lim) s[j] = -INFINITY;
            }
            float mx = max3(s[0], s[1], s[2]), mx2 = max3(s[3], s[4], s[5]);
#pragma unroll
            for (int j = 6; j < 126; j += 4) {
                mx = max3(mx, s[j], s[j + 1]);
                mx2 = max3(mx2, s[j + 2], s[j + 3]);
            }
            mx = max3(mx, s[126], s[127]);
            mx = fmaxf(mx, mx2) * sc;
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
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tc::tmem_ld32_raw(to + c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tc::tmem_st32_raw(to + c, o);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            const uint64_t sc2 = pack2(sc, sc), nb2 = pack2(-base, -base);
            uint64_t sum = 0;
#pragma unroll
            for (int c = 0; c < 128; c += 64) {
                uint32_t p[32];
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float e0, e1;
                    unpack2(fma2(pack2(s[c + j], s[c + j + 1]), sc2, nb2), e0, e1);
                    if (masked) {                    // exact zeros where masked
                        e0 = j0 + c + j > lim ? 0.f : exp2_sfu(e0);
                        e1 = j0 + c + j + 1 > lim ? 0.f : exp2_sfu(e1);
                    } else if ((j & 7) == 6) {
                        exp2_poly(e0, e1);
                    } else {
                        e0 = exp2_sfu(e0);
                        e1 = exp2_sfu(e1);
                    }
                    sum = add2(sum, pack2(e0, e1));
                    p[j / 2] = pack_bf16(e0, e1);
                }
                tc::tmem_st32_raw(ts + c / 2, p);
            }
            float s0, s1;
            unpack2(sum, s0, s1);
            l += s0 + s1;
            if (clears && i + 1 == it.total && kv_end - j0 < kKeys) {
                // values that no row of the block sees may be anything: clear them
                const int t = 2 * i + 1, slot = t % C::kRing;
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&kv_full[slot], (uint32_t)((t / C::kRing) & 1)));
                if (!ok) break;
                uint8_t* v = ring + slot * C::kTile;
                const int first = kv_end - j0;
                for (int e = (warp & 3) * 32 + lane; e < (kKeys - first) * 8 * C::kHalves; e += 128) {
                    const int r = first + e / (8 * C::kHalves), c = e % (8 * C::kHalves);
                    *reinterpret_cast<uint4*>(v + (c >> 3) * C::kHalf + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_async_smem();
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&p_full[x]);
        }
        if (steps > 0 && ok) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&o_full[x], 0));
            tc::tc_fence_after();
        }
        if (!ok && lane == 0) s_timeout = 1;
        if (ok) {
            const bool empty = lim < 0;
            const float inv = empty ? 0.f : 1.0f / l;
            const int64_t at = (((int64_t)it.sq.q0 + it.tok[x] + tok) * a.HQ + it.kvh * G + (row - tok * G)) * D;
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
            if (!finite && live) s_redo = 1;
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
    if (tid == 0) {
        if (s_timeout) atomicMax(&g_attn_tc_error, GDN_DEVERR_TIMEOUT);
        // tiles of a bad table may be listed twice: never past the list's end
        if (s_redo) {
            const int at = atomicAdd(&plan.counts[1], 1);
            if (at < plan.max_redo) plan.redo[at] = make_int4(pt.x, pt.y, it.kvh, 0);
        }
    }
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    using C = Cfg<D>;
    const int G = a.HQ / a.HKV, tokens = kRows / G;
    const AttnPlan plan = attn_plan(a.ws, a.n_tokens, a.n_seqs, a.HKV, 1, 2 * tokens);
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
    attn_prefill_kernel<D><<<(unsigned)(plan.max_tiles * a.HKV), kThreads, C::kSmem, s>>>(tq, tk, tv, a, plan, tokens,
                                                                                         box_rows);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_attn_redo(a, plan, 2 * tokens, s);
}

}  // namespace

bool attn_tc_supported(int HQ, int HKV) { return HQ / HKV <= kRows; }

size_t attn_tc_bytes(int64_t n_tokens, int n_seqs, int HQ, int HKV) {
    const AttnPlan p = attn_plan(nullptr, n_tokens, n_seqs, HKV, 1, 2 * (kRows / (HQ / HKV)));
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
