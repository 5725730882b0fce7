// attn_decode.cu -- one new token per sequence, or a short piece of them, attends to its pages of the
// key-value cache.
//
//   o_h = sum_j w_j v_j / sum_j w_j,   w_j = e^{scale q_h . k_j - m},  j over the context.
//
// Bound: HBM.  Every key and value is read once for the whole group of query heads that share
// it; two FLOPs per byte and query head, so even a group of 16 leaves the arithmetic far below
// the tensor cores' reach.  What decides the time is how many bytes each SM keeps in flight and
// how evenly the contexts, which are ragged, spread over the SMs.
//
// Split.  The work is one list of tiles of KT keys: sequence by sequence, key-value head by
// head, tile by tile.  The grid is one block per SM; block c takes the tiles from c N / grid to
// (c + 1) N / grid, so every block reads the same number of bytes whatever the lengths are.  A
// block's range may begin and end inside a (sequence, head) item; those pieces leave their
// running maximum, sum and unnormalised output in the workspace, two slots a block, and a second
// small kernel joins them in the order of the blocks (the result does not depend on timing).
// Lengths live on the device: each block finds its range by a scan over them.
//
// An item's start and end count as a few tiles in the split.
//
// Measured: 64 ragged contexts to 32K, 8 key-value heads, gated: 550 us for 3.75 GB (6.8 TB/s; 630 us in
// long runs, where the power limit holds the clock at 1.7 GHz); one context of 262K, 2 heads: 50 us for
// 268 MB; of 1000: 10 us, the chain of lengths, table, tile and join; fp32, 24 contexts, 64 wide: 71 us
// for 323 MB.
//
// Short pieces (P): the rows are a piece's (token, head) pairs, 16 at most, each with a last key of its
// own.  Values that only some rows see stay in shared memory; one that is not finite shows in the other
// rows' outputs, and those rows are listed for the pass that leaves masked places out.
//
// Block: a producer warp copies tiles into a ring in shared memory by TMA, 128B-swizzled, one
// box per page part (rows of a token's head are 128 or 256 bytes, heads and tokens strided);
// eight consumer warps in teams of two or four take the tiles in turn, a warp a fixed share of
// a tile's keys, each with its own running statistics, so that teams only meet at the end of an item.
//   bf16: mma.sync m16n8k16 with the group's heads as M (up to 16), the fragments read by
//     ldmatrix; tcgen05 would need 128 rows and has nothing to gain on a tile read once.
//   fp32: CUDA cores (no TF32), a lane a quarter of a key's elements for the scores, D / 32
//     output columns a lane for the values.
#include "attn_common.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

using bf16 = __nv_bfloat16;

__device__ int g_decode_attn_error;

constexpr int kWarps = 8, kConsumers = kWarps * 32, kThreads = kConsumers + 32;
constexpr int kMaxGrid = 192;             // blocks, for the workspace size
constexpr float kLog2e = 1.4426950408889634f;

// R: query heads a block serves at once (rows of the statistics).
template <typename IO, int D, int R>
struct Cfg {
    static constexpr int KT = 16384 / (D * (int)sizeof(IO));        // keys per tile: 32 KB of keys and values
    static constexpr int TW = KT < 64 ? KT / 16 : 4;                // warps of a team, which share a tile
    static constexpr int Teams = kWarps / TW;
    static constexpr int KW = KT / TW;                              // keys per warp: 16, or 32 (bf16, D = 64)
    static constexpr int NB = D * (int)sizeof(IO) / 128;            // 128-byte column blocks
    static constexpr int kBlk = KT * 128;                           // bytes of one column block
    static constexpr int kStage = 2 * NB * kBlk;                    // keys, then values
    static constexpr int kMerge = 8 * R * (D + 4) * 4;              // the warps' outputs at an item's end
    static constexpr int kQ = sizeof(IO) == 4 ? R * D * 4 : 0;      // fp32: the rows' queries
    static constexpr int kFit = (226 * 1024 - 1024 - kMerge - kQ) / kStage;
    // ring slots, a multiple of the teams: a slot then always belongs to the same team, which waits
    // for every phase of its barrier
    static constexpr int kStages = kFit / Teams * Teams;
    static constexpr int kSmem = kStages * kStage + kMerge + kQ + 1024;
    // What an item's start and end cost a block (its queries' way, the joining of its warps, about
    // 2 us), in tiles.  It is counted in the split: 24 ragged contexts in fp32, 16 heads: 100 us
    // without, 70 us with it.
    static constexpr int kItemCost = 4;
};

// The context that the kernel reads for a sequence: P, only where the sequence has a short piece.
template <bool P>
__device__ __forceinline__ int keys_of(const AttnArgs& a, const SeqRows& r) {
    return !P || short_piece(a, r) ? r.n_kv : 0;
}
template <bool P>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int n, int kt, int* bad) {
    const SeqRows r = seq_rows(a, n);
    if (r.bad) *bad = r.bad;
    return (keys_of<P>(a, r) + kt - 1) / kt;
}
// Where row r of an item is in q, z and o: P, the rows are the piece's (token, query head) pairs.
template <bool P>
__device__ __forceinline__ int64_t row_at(const AttnArgs& a, int D, int r) {
    if constexpr (!P) return (int64_t)r * D;
    const int G = a.HQ / a.HKV, t = r / G;
    return ((int64_t)t * a.HQ + (r - t * G)) * D;
}

// Units of work of sequence n: per head (and row block) its tiles, one unit each, and in front of
// them the item's cost.  Tile t of an item that begins at unit u is unit u + kItemCost + t; a block
// has the tiles whose units are in its share.
template <typename C, bool P>
__device__ __forceinline__ int64_t cost_of(const AttnArgs& a, int n, int subs, int* bad) {
    const int tiles = tiles_of<P>(a, n, C::KT, bad);
    return tiles > 0 ? (int64_t)(tiles + C::kItemCost) * subs : 0;
}

// Block-wide: the total of per(n) over all sequences, the blocks that share it (no more than there
// are units, so that none is empty), and the sequence that holds block c's first unit with the
// units before it (n = -1: block c has none).
struct Place {
    int64_t total, before, at;
    int n, blocks;
};
template <typename F>
__device__ Place find_place(int n_seqs, F per, int c, int grid, int64_t* s_warp, Place* s_out) {
    // thread t owns the sequences [t k, (t + 1) k)
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, nw = blockDim.x >> 5;
    const int k = (n_seqs + blockDim.x - 1) / blockDim.x;
    const int lo = min(tid * k, n_seqs), hi = min(lo + k, n_seqs);
    int64_t sum = 0;
    for (int n = lo; n < hi; ++n) sum += per(n);
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[w] = incl;
    if (tid == 0) s_out->n = -1;
    __syncthreads();
    int64_t base = 0, total = 0;
    for (int i = 0; i < nw; ++i) {
        if (i < w) base += s_warp[i];
        total += s_warp[i];
    }
    const int blocks = (int)min((int64_t)grid, total);
    const int64_t at = c < blocks ? total * c / blocks : total;
    int64_t before = base + incl - sum;
    if (at >= before && at < before + sum) {
        for (int n = lo; n < hi; ++n) {
            const int64_t u = per(n);
            if (at < before + u) {
                s_out->n = n;
                s_out->before = before;
                break;
            }
            before += u;
        }
    }
    __syncthreads();
    Place p = *s_out;
    p.total = total;
    p.at = at;
    p.blocks = blocks;
    return p;
}

struct Partials {
    int4* desc;           // [grid]  {first, last block of the item that block c began inside, as the first that did,
                          //          or first = -1; sequence; first query head}
    float* o;             // [grid][2][R][D]
    float2* ml;           // [grid][2][R]  (m in log2 units, l)
};
__host__ __device__ inline Partials partials(void* ws, int R, int D) {
    Partials p;
    p.desc = reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + kStatusBytes);
    p.ml = reinterpret_cast<float2*>(p.desc + kMaxGrid);
    p.o = reinterpret_cast<float*>(p.ml + kMaxGrid * 2 * R);
    return p;
}

// ---- a warp's running state over the keys it takes ----------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}

template <typename IO, int D, int R, bool P>
struct Warp;

// bf16: rows are heads (P: a piece's (token, head) pairs), 16 of them; a thread holds rows lane / 4 and
// lane / 4 + 8.
template <int D, bool P>
struct Warp<bf16, D, 16, P> {
    using C = Cfg<bf16, D, 16>;
    uint32_t q[D / 16][4];
    float o[D / 8][4];
    float m[2], l[2];

    __device__ __forceinline__ void start(const AttnArgs& a, const bf16* qrow, int rows) {
        const int lane = threadIdx.x & 31, r = lane >> 2, c = (lane & 3) * 2;
        const bf16 *p0 = qrow + row_at<P>(a, D, r) + c, *p1 = qrow + row_at<P>(a, D, r + 8) + c;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            q[k][0] = r < rows ? *reinterpret_cast<const uint32_t*>(p0 + k * 16) : 0u;
            q[k][1] = r + 8 < rows ? *reinterpret_cast<const uint32_t*>(p1 + k * 16) : 0u;
            q[k][2] = r < rows ? *reinterpret_cast<const uint32_t*>(p0 + k * 16 + 8) : 0u;
            q[k][3] = r + 8 < rows ? *reinterpret_cast<const uint32_t*>(p1 + k * 16 + 8) : 0u;
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    // the warp's KW keys, rows KW w .. of the tile, of which the first `valid` exist (> 0); P: the first
    // `all` of which every row sees, a row of token t those up to all + t
    __device__ __forceinline__ void step(const AttnArgs& a, uint8_t* tile, int w, int valid, int all, float sc,
                                         const float*) {
        constexpr int NS = C::KW / 16;
        const int lane = threadIdx.x & 31;
        uint8_t* vt = tile + C::NB * C::kBlk;
        if (valid < C::KW) {    // values past the context may be anything: 0 * NaN must not enter
            for (int i = lane; i < (C::KW - valid) * C::NB * 8; i += 32) {
                const int row = C::KW * w + valid + i / (C::NB * 8), c = i % (C::NB * 8);
                *reinterpret_cast<uint4*>(vt + (c >> 3) * C::kBlk + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            tc::fence_async_smem();        // before the ring slot's next copy overwrites them
            __syncwarp();
        }
        const uint32_t kb = tc::smem_u32(tile), vb = tc::smem_u32(vt);
        const int mat = lane >> 3, mr = lane & 7;
        float s[2 * NS][4] = {};
        {   // matrices: keys 0-7 and 8-15 (mat >> 1), element halves (mat & 1)
            const int row = C::KW * w + ((mat >> 1) << 3) + mr;
            const uint32_t base = kb + row * 128;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const int chunk = (k & 3) * 2 + (mat & 1);
                const uint32_t at = base + (k >> 2) * C::kBlk + ((chunk ^ mr) << 4);
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    uint32_t b[4];
                    ldsm4(at + n * 16 * 128, b);
                    mma16816(s[2 * n], q[k], b[0], b[1]);
                    mma16816(s[2 * n + 1], q[k], b[2], b[3]);
                }
            }
        }
        // the reference m moves only when a score exceeds it by more than 2^8 (weights stay below
        // that), so that a step usually needs no reduction over the row's four threads
        bool grow = false;
        int sees[2] = {valid, valid};
        if (P && all < valid) {
            // (0 * v is not 0 where a value that the row does not see is not finite: that shows in the
            // output, and the row is done again)
            const int G = a.HQ / a.HKV;
            sees[0] = min(valid, all + (lane >> 2) / G);
            sees[1] = min(valid, all + ((lane >> 2) + 8) / G);
        }
#pragma unroll
        for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = j * 8 + (lane & 3) * 2 + (i & 1);
                s[j][i] = key < sees[i >> 1] ? s[j][i] * sc : -INFINITY;
                grow = grow || s[j][i] > m[i >> 1] + 8.f;
            }
        if (__any_sync(0xffffffffu, grow)) {
            float al[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = m[r];
#pragma unroll
                for (int j = 0; j < 2 * NS; ++j) mx = fmaxf(mx, fmaxf(s[j][2 * r], s[j][2 * r + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                al[r] = mx == -INFINITY ? 1.f : exp2f(m[r] - mx);
                m[r] = mx;
                l[r] *= al[r];
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][0] *= al[0];
                o[j][1] *= al[0];
                o[j][2] *= al[1];
                o[j][3] *= al[1];
            }
        }
        const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
        for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[j][i] = exp2f(s[j][i] - base[i >> 1]);
                l[i >> 1] += s[j][i];
            }
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            // the weights are rounded to bf16 for the product (half a step, 2^-8, each); their sum is not
            const uint32_t p[4] = {pack_bf16(s[2 * n][0], s[2 * n][1]), pack_bf16(s[2 * n][2], s[2 * n][3]),
                                   pack_bf16(s[2 * n + 1][0], s[2 * n + 1][1]),
                                   pack_bf16(s[2 * n + 1][2], s[2 * n + 1][3])};
            // matrices: keys 0-7 and 8-15 (mat & 1), column eights (mat >> 1)
            const int row = C::KW * w + 16 * n + ((mat & 1) << 3) + mr;
            const uint32_t base_v = vb + row * 128;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                uint32_t b[4];
                const int chunk = (c & 3) * 2 + (mat >> 1);
                ldsm4t(base_v + (c >> 2) * C::kBlk + ((chunk ^ mr) << 4), b);
                mma16816(o[2 * c], p, b[0], b[1]);
                mma16816(o[2 * c + 1], p, b[2], b[3]);
            }
        }
    }

    // to shared memory: o rows of D + 4 floats, (m, l) after the columns
    __device__ __forceinline__ void put(float* out, int rows) {
        const int lane = threadIdx.x & 31, r = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const int row = r + 8 * h;
            if (row < rows) {
                float* p = out + row * (D + 4);
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    *reinterpret_cast<float2*>(p + j * 8 + c) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
                if ((lane & 3) == 0) *reinterpret_cast<float2*>(p + D) = make_float2(m[h], l[h]);
            }
        }
    }
};

// fp32: a lane holds D / 32 columns of every row's output; the scores of key 8 s + lane / 4 of the
// warp's keys are summed by its four lanes.  The reference m moves only when a score exceeds it by
// more than 2^8 (weights stay below that), so that a step usually needs no reduction over the
// warp; l is a lane's own sum over its keys until the end.
template <int D, int R>
struct Warp<float, D, R, false> {
    using C = Cfg<float, D, R>;
    static constexpr int E = D / 32, NS = C::KW / 8;
    float o[R][E];
    float m[R], l[R];

    __device__ __forceinline__ void start(const AttnArgs&, const float*, int) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[r][e] = 0.f;
        }
    }

    __device__ __forceinline__ void step(const AttnArgs&, uint8_t* tile, int w, int valid, int, float sc,
                                         const float* sq) {
        const int lane = threadIdx.x & 31, key = lane >> 2, part = lane & 3;
        const uint8_t* vt = tile + C::NB * C::kBlk;
        float s[NS][R];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int r = 0; r < R; ++r) s[n][r] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const int c = part + 4 * i;                       // 16-byte chunk of the row
            float4 k[NS];
#pragma unroll
            for (int n = 0; n < NS; ++n)                      // (rows 8 apart: the same swizzle)
                k[n] = *reinterpret_cast<const float4*>(tile + (c >> 3) * C::kBlk + (C::KW * w + 8 * n + key) * 128 +
                                                        (((c & 7) ^ key) << 4));
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 q = *reinterpret_cast<const float4*>(sq + r * D + 4 * c);
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    s[n][r] = fmaf(k[n].x, q.x, fmaf(k[n].y, q.y, fmaf(k[n].z, q.z, fmaf(k[n].w, q.w, s[n][r]))));
            }
        }
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float y = s[n][r];
                y += __shfl_xor_sync(0xffffffffu, y, 1);
                y += __shfl_xor_sync(0xffffffffu, y, 2);
                y = 8 * n + key < valid ? y * sc : -INFINITY;
                grow = grow || y > m[r] + 8.f;
                s[n][r] = y;
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float mx = s[0][r];
                if constexpr (NS == 2) mx = fmaxf(mx, s[1][r]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                mx = fmaxf(mx, m[r]);
                const float al = mx == -INFINITY ? 1.f : exp2f(m[r] - mx);
                m[r] = mx;
                l[r] *= al;
#pragma unroll
                for (int e = 0; e < E; ++e) o[r][e] *= al;
            }
        }
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s[n][r] = exp2f(s[n][r] - (m[r] == -INFINITY ? 0.f : m[r]));
                l[r] += s[n][r];
            }
#pragma unroll
        for (int j = 0; j < C::KW; ++j) {
            if (j < valid) {                   // values past the context never enter
                float v[E];
                const int c = lane * E / 4;    // this lane's columns: E consecutive floats
                const uint8_t* p = vt + (c >> 3) * C::kBlk + (C::KW * w + j) * 128 + (((c & 7) ^ (j & 7)) << 4);
                if constexpr (E == 4) {
                    *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p);
                } else {
                    *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(p + (lane & 1) * 8);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float pr = __shfl_sync(0xffffffffu, s[j >> 3][r], (j & 7) * 4);
#pragma unroll
                    for (int e = 0; e < E; ++e) o[r][e] = fmaf(pr, v[e], o[r][e]);
                }
            }
        }
    }

    __device__ __forceinline__ void put(float* out, int rows) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 4);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 8);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
            if (r < rows) {
                float* p = out + r * (D + 4);
#pragma unroll
                for (int e = 0; e < E; ++e) p[lane * E + e] = o[r][e];
                if (lane == 0) *reinterpret_cast<float2*>(p + D) = make_float2(m[r], l[r]);
            }
        }
    }
};

// Where a block is in its share: sequence, (head, row block) of it, tile of that item, the tile's
// unit.
struct Cursor {
    int n, sub, tile, tiles, len, q0, n_q;
    int64_t unit;
};
template <typename C, bool P>
__device__ __forceinline__ void cursor_load(const AttnArgs& a, Cursor& c) {
    while (true) {      // (the last sequence ends the search, tiles or not)
        const SeqRows r = seq_rows(a, c.n);
        c.len = keys_of<P>(a, r);
        c.tiles = (c.len + C::KT - 1) / C::KT;
        c.q0 = r.q0;
        c.n_q = r.n_q;
        if (c.tiles > 0 || c.n + 1 >= a.n_seqs) return;
        ++c.n;
    }
}
// To the next tile; false if it is not in the block's share, which ends before unit `end`.
template <typename C, bool P>
__device__ __forceinline__ bool cursor_next(const AttnArgs& a, Cursor& c, int subs, int64_t end) {
    ++c.unit;
    if (++c.tile < c.tiles) return c.unit < end;
    c.unit += C::kItemCost;
    if (c.unit >= end) return false;
    c.tile = 0;
    if (++c.sub == subs) {
        c.sub = 0;
        if (++c.n >= a.n_seqs) return false;
        cursor_load<C, P>(a, c);
    }
    return true;
}

// P: short pieces of prompts instead of one token per sequence (bf16, one row block: hb = 1).
template <typename IO, int D, int R, bool P>
__global__ void __launch_bounds__(kThreads, 1) attn_decode_kernel(const __grid_constant__ CUtensorMap tk,
                                                                  const __grid_constant__ CUtensorMap tv, AttnArgs a,
                                                                  int hb, AttnPlan plan) {
    using C = Cfg<IO, D, R>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t s_warp[kThreads / 32];
    __shared__ Place s_place;
    __shared__ __align__(8) uint64_t full[S], empty[S];
    __shared__ int s_dead, s_redo;
    // ring tiles 1024-byte aligned (the swizzle's period)
    uint8_t* ring = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    float* merge = reinterpret_cast<float*>(ring + S * C::kStage);
    float* sq = merge + C::kMerge / 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.HQ / a.HKV, subs = a.HKV * hb;

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], C::TW);
        }
        tc::fence_mbar_init();
        s_dead = s_redo = 0;
    }
    tc::grid_dependency_sync();
    int bad = 0;
    const Place pl = find_place(
        a.n_seqs, [&](int n) { return cost_of<C, P>(a, n, subs, &bad); }, blockIdx.x, gridDim.x, s_warp, &s_place);
    if (bad && blockIdx.x == 0) atomicMax(&g_decode_attn_error, bad);
    // contexts of no keys: zeros, a sequence's rows by one block
    for (int n = blockIdx.x; n < a.n_seqs; n += gridDim.x) {
        const SeqRows r = seq_rows(a, n);
        if (!r.bad && r.n_kv == 0 && (!P || short_piece(a, r)))
            for (int i = tid; i < r.n_q * a.HQ * D; i += kThreads)
                store_elem((IO*)a.o, (int64_t)r.q0 * a.HQ * D + i, 0.f);
    }
    const Partials part = partials(a.ws, R, D);
    if (tid == 0) {      // for the join
        int4 d = make_int4(-1, 0, 0, 0);
        if (pl.n >= 0) {
            const int tiles = tiles_of<P>(a, pl.n, C::KT, &bad);
            const int sub = (int)((pl.at - pl.before) / (tiles + C::kItemCost));
            // unit of the item's first tile, and the blocks that hold its tiles: unit u is in the
            // last block that begins at or before it
            const int64_t t0 = pl.before + (int64_t)sub * (tiles + C::kItemCost) + C::kItemCost, N = pl.total;
            const int c0 = (int)(((t0 + 1) * pl.blocks - 1) / N);
            if (pl.at > t0 && (int)blockIdx.x == c0 + 1)
                d = make_int4(c0, (int)(((t0 + tiles) * pl.blocks - 1) / N), pl.n, sub / hb * G + sub % hb * R);
        }
        part.desc[blockIdx.x] = d;
    }
    if (pl.n < 0) return;

    const int64_t end = pl.total * (blockIdx.x + 1) / pl.blocks;
    Cursor cur;
    cur.n = pl.n;
    cursor_load<C, P>(a, cur);
    {
        const int64_t in_seq = pl.at - pl.before;
        cur.sub = (int)(in_seq / (cur.tiles + C::kItemCost));
        const int u = (int)(in_seq - (int64_t)cur.sub * (cur.tiles + C::kItemCost));
        cur.tile = max(u - C::kItemCost, 0);
        cur.unit = pl.at + max(C::kItemCost - u, 0);
    }
    if (cur.unit >= end) return;       // the share ends within an item's cost: no tile
    const int rows_box = min(1 << a.kv.page_shift, C::KT);

    if (warp == kConsumers / 32) {
        // ---- producer: lane (g, kind, block) issues one box of the tile
        const int boxes = C::KT / rows_box;
        const int lg = lane / (2 * C::NB), lk = (lane / C::NB) & 1, lb = lane % C::NB;
        const int64_t none = (int64_t)a.kv.n_pages << a.kv.page_shift;        // a row past the cache: zero fill
        int ent = 0, ent_n = -1, ent_base = 0;      // 32 table entries, one a lane
        bool ok = true;
        bool more = true;
        for (int it = 0; more; ++it) {
            const int st = it % S;
            const uint32_t ph = (uint32_t)((it / S) & 1);
            if (it >= S && ok) {
                ok = tc::mbar_wait(&empty[st], ph ^ 1);
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!ok) break;
            const int pos0 = cur.tile * C::KT;
            const int first = pos0 >> a.kv.page_shift;
            const int last = min(pos0 + C::KT, cur.len) - 1;
            if (cur.n != ent_n || first < ent_base || (last >> a.kv.page_shift) >= ent_base + 32) {
                ent_n = cur.n;
                ent_base = first;
                ent = 0;
                if (ent_base + lane <= ((cur.len - 1) >> a.kv.page_shift))
                    ent = a.kv.table[(int64_t)cur.n * a.kv.max_pages + ent_base + lane];
            }
            const int kvh = cur.sub / hb;
            const int groups = min(boxes, (last - pos0) / rows_box + 1);
            const int pos = pos0 + lg * rows_box;
            const int page = __shfl_sync(0xffffffffu, ent, min(max((pos >> a.kv.page_shift) - ent_base, 0), 31));
            uint8_t* tile = ring + st * C::kStage;
            if (lane == 0) tc::mbar_expect_tx(&full[st], (uint32_t)(groups * rows_box * 128 * 2 * C::NB));
            __syncwarp();
            if (lg < groups) {
                int64_t row = none;
                if (page >= 0 && page < a.kv.n_pages)
                    row = ((int64_t)page << a.kv.page_shift) + (pos & ((1 << a.kv.page_shift) - 1));
                else
                    atomicMax(&g_decode_attn_error, GDN_DEVERR_PAGE);
                tc::tma_load_3d(tile + (lk * C::NB + lb) * C::kBlk + lg * rows_box * 128, lk ? &tv : &tk, &full[st],
                                lb * (128 / (int)sizeof(IO)), kvh, (int)row);
            }
            more = cursor_next<C, P>(a, cur, subs, end);
        }
        if (!ok) {      // an expired wait: let every copy that was issued land before leaving
            if (lane == 0) atomicMax(&g_decode_attn_error, GDN_DEVERR_TIMEOUT);
            for (int i = 0; i < S; ++i) tc::mbar_wait(&full[i], 0, 1000000);
        }
        return;
    }

    // ---- consumers
    const int team = warp / C::TW, w = warp % C::TW;
    Warp<IO, D, R, P> st;
    const float sc = a.scale * kLog2e;
    bool ok = true, fresh = true, from_start = false, more = true;
    for (int it = 0; more; ++it) {
        const int kvh = cur.sub / hb, h0 = kvh * G + (cur.sub - kvh * hb) * R;
        const int rows = P ? cur.n_q * G : min(R, (kvh + 1) * G - h0);
        const int64_t qrow = ((int64_t)cur.q0 * a.HQ + h0) * D;
        if (fresh) {
            from_start = cur.tile == 0;
            if constexpr (sizeof(IO) == 4) {
                // the rows' queries for every warp (rows past the group: zeros)
                for (int i = tid; i < R * D; i += kConsumers)
                    sq[i] = i < rows * D ? ((const float*)a.q)[qrow + i] : 0.f;
                tc::named_bar(1, kConsumers);
            }
            st.start(a, (const IO*)a.q + qrow, rows);
            fresh = false;
        }
        if (it % C::Teams == team) {
            const int s = it % S;
            if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[s], (uint32_t)((it / S) & 1)));
            const int left = cur.len - cur.tile * C::KT - w * C::KW, valid = min(C::KW, left);
            if (ok && valid > 0) st.step(a, ring + s * C::kStage, w, valid, left - cur.n_q + 1, sc, sq);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[s]);
        }
        const bool item_end = cur.tile + 1 == cur.tiles;
        const int n = cur.n, past = cur.len - cur.n_q;
        more = cursor_next<C, P>(a, cur, subs, end);
        if (item_end || !more) {
            // the segment is over: join the eight warps
            if (!ok && lane == 0) s_dead = 1;
            st.put(merge + warp * R * (D + 4), rows);
            tc::named_bar(1, kConsumers);
            const bool whole = from_start && item_end;
            const int64_t slot = (int64_t)blockIdx.x * 2 + (from_start ? 1 : 0);
            for (int i = tid; i < rows * (D / 4); i += kConsumers) {
                const int r = i / (D / 4), c = (i % (D / 4)) * 4;
                const float* p = merge + r * (D + 4);
                float m = -INFINITY, l = 0.f;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < 8; ++k) m = fmaxf(m, p[k * R * (D + 4) + D]);
                const float base = m == -INFINITY ? 0.f : m;
                for (int k = 0; k < 8; ++k) {
                    // (a warp that took no key has m = -inf, l = 0, o = 0: it adds zeros; one whose keys all
                    // score -inf may hold NaN, from values that are not finite, and hands them on)
                    const float* pk = p + k * R * (D + 4);
                    const float f = exp2f(pk[D] - base);
                    const float4 y = *reinterpret_cast<const float4*>(pk + c);
                    l = fmaf(f, pk[D + 1], l);
                    x.x = fmaf(f, y.x, x.x);
                    x.y = fmaf(f, y.y, x.y);
                    x.z = fmaf(f, y.z, x.z);
                    x.w = fmaf(f, y.w, x.w);
                }
                if (whole) {
                    const bool none = P && past < 0 && past + r / G < 0;             // the row sees no key
                    const float inv = 1.0f / l;
                    const float y[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
                    const int64_t at = qrow + row_at<P>(a, D, r) + c;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float out = none ? 0.f : y[e];
                        if constexpr (P)
                            if (!(fabsf(out) <= 3.4028235e38f)) s_redo = 1;
                        if (a.z && !none) out = gate_out(out, load_elem((const IO*)a.z, at + e));
                        store_elem((IO*)a.o, at + e, out);
                    }
                } else {
                    *reinterpret_cast<float4*>(part.o + (slot * R + r) * D + c) = x;
                    if (c == 0) part.ml[slot * R + r] = make_float2(m, l);
                }
            }
            tc::named_bar(1, kConsumers);
            if constexpr (P)
                if (tid == 0 && s_redo) {
                    list_redo(plan, n, kvh, 0, rows);
                    s_redo = 0;          // (set again only after the next item's first barrier)
                }
            fresh = true;
        }
    }
    if (s_dead && tid == 0) atomicMax(&g_decode_attn_error, GDN_DEVERR_TIMEOUT);
}

// Joins the pieces of the items that more than one block took: of the item that block c of the first
// kernel left to it.  Many pieces (a long context over many blocks): block (c - 1, r) is row r, a warp
// takes every eighth piece.  At most kBatch: block (c - 1, y) is rows 8 y .. 8 y + 7, a warp each, and
// the other y have nothing to do (16 rows of 512 items: 4 against 12 us).  All of a warp's loads
// are in flight at once, kBatch at a time.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kBatch = 8;
template <int E> struct Vec;
template <> struct Vec<2> { using T = float2; };
template <> struct Vec<4> { using T = float4; };
template <typename IO, int D, int R, bool P>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(AttnArgs a, AttnPlan plan) {
    constexpr int E = D / 32;
    __shared__ float s_o[kJoinWarps][D];
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    tc::grid_dependency_sync();
    const Partials part = partials(a.ws, R, D);
    const int4 d = part.desc[blockIdx.x + 1];
    const int first = d.x, last = d.y, G = a.HQ / a.HKV;
    if (first < 0) return;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const bool few = last - first < kBatch;
    const int r = few ? blockIdx.y * kJoinWarps + w : blockIdx.y;
    if (few && blockIdx.y * kJoinWarps >= R) return;
    const SeqRows sr = P ? seq_rows(a, d.z) : SeqRows{d.z, 1, 0, 0};
    if (P ? r >= sr.n_q * G : (r >= R || d.w % G + r >= G)) return;          // (a warp, or the block)
    const int start = few ? first : first + w, stride = few ? 1 : kJoinWarps;
    auto slot = [&](int b) { return ((int64_t)b * 2 + (b == first ? 1 : 0)) * R + r; };
    float m = -INFINITY, l = 0.f, x[E] = {};
    for (int b0 = start; b0 <= last; b0 += kBatch * stride) {
        float2 ml[kBatch];
        typename Vec<E>::T y[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int b = min(b0 + i * stride, last);          // (past the end: read again, not used)
            ml[i] = part.ml[slot(b)];
            y[i] = reinterpret_cast<const typename Vec<E>::T*>(part.o + slot(b) * D)[lane];
        }
        float mn = m;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) mn = fmaxf(mn, ml[i].x);
        const float base = mn == -INFINITY ? 0.f : mn, g = exp2f(m - base);
        m = mn;
        l *= g;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= g;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (b0 + i * stride <= last) {
                const float f = exp2f(ml[i].x - base);
                const float* v = reinterpret_cast<const float*>(&y[i]);
                l = fmaf(f, ml[i].y, l);
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = fmaf(f, v[e], x[e]);
            }
    }
    const bool none = P && sr.n_kv - sr.n_q + r / G < 0;         // the row sees no key
    const int64_t at = ((int64_t)sr.q0 * a.HQ + d.w) * D + row_at<P>(a, D, r);
    // column c of the row; whether it is finite
    auto put = [&](int c, float y) {
        if (none) y = 0.f;
        store_elem((IO*)a.o, at + c, a.z && !none ? gate_out(y, load_elem((const IO*)a.z, at + c)) : y);
        return fabsf(y) <= 3.4028235e38f;
    };
    bool finite = true;
    if (few) {
#pragma unroll
        for (int e = 0; e < E; ++e) finite = put(lane * E + e, x[e] / l) && finite;
        if (P && !__all_sync(0xffffffffu, finite) && lane == 0) list_redo(plan, d.z, d.w / G, r, 1);
        return;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[w][lane * E + e] = x[e];
    if (lane == 0) {
        s_m[w] = m;
        s_l[w] = l;
    }
    __syncthreads();
    if (tid < D) {
        m = s_m[0];
#pragma unroll
        for (int i = 1; i < kJoinWarps; ++i) m = fmaxf(m, s_m[i]);
        const float base = m == -INFINITY ? 0.f : m;
        float y = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) {
            const float f = exp2f(s_m[i] - base);
            y = fmaf(f, s_o[i][tid], y);
            sum = fmaf(f, s_l[i], sum);
        }
        finite = put(tid, y / sum);
    }
    if constexpr (P)
        if (__syncthreads_or(!finite) && tid == 0) list_redo(plan, d.z, d.w / G, r, 1);
}

template <typename IO, int D, int R, bool P = false>
cudaError_t launch(const AttnArgs& a, cudaStream_t s, const AttnPlan& plan = AttnPlan{}) {
    using C = Cfg<IO, D, R>;
    static_assert(C::kStages >= 4 && C::kSmem <= 226 * 1024, "decode: shared memory");
    const int G = a.HQ / a.HKV, hb = (G + R - 1) / R;          // (P: 1)
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // one block per SM, fewer where the longest contexts the tables can hold have fewer tiles
    const int64_t longest = (((int64_t)a.kv.max_pages << a.kv.page_shift) + C::KT - 1) / C::KT;
    const int64_t most = (int64_t)a.n_seqs * a.HKV * hb * longest;
    int grid = sms < kMaxGrid ? sms : kMaxGrid;
    if (most < grid) grid = most > 0 ? (int)most : 1;
    CUtensorMap tk, tv;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.HKV, (cuuint64_t)a.kv.n_pages << a.kv.page_shift};
    const cuuint64_t str[2] = {(cuuint64_t)D * sizeof(IO), (cuuint64_t)a.HKV * D * sizeof(IO)};
    const int page = 1 << a.kv.page_shift;
    const cuuint32_t box[3] = {(cuuint32_t)(128 / sizeof(IO)), 1, (cuuint32_t)(page < C::KT ? page : C::KT)};
    const CUtensorMapDataType dt = sizeof(IO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    // a head's row of 128 bytes has another head's beside it, which this block does not read next
    const CUtensorMapL2promotion l2 =
        D * sizeof(IO) == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    if (!make_map(&tk, dt, a.kv.k, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B, l2) ||
        !make_map(&tv, dt, a.kv.v, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B, l2))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    e = allow_smem((const void*)attn_decode_kernel<IO, D, R, P>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attn_decode_kernel<IO, D, R, P>, dim3((unsigned)grid), dim3(kThreads), C::kSmem, s, tk, tv, a, hb,
                   plan);
    if (e != cudaSuccess) return e;
    count_launch();
    if (grid == 1) return cudaSuccess;           // nothing to join
    const int64_t rows = P ? a.n_tokens * G : G;              // the most that an item can have
    e = launch_pdl(attn_join_kernel<IO, D, R, P>, dim3((unsigned)(grid - 1), (unsigned)(rows < R ? rows : R)),
                   dim3(kJoinThreads), 0, s, a, plan);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <int D>
cudaError_t launch_f32(const AttnArgs& a, cudaStream_t s) {
    // rows cost registers and work in the fp32 kernel, used or not: the smallest count that holds
    // the group, at most 8
    const int G = a.HQ / a.HKV;
    if (G == 1) return launch<float, D, 1>(a, s);
    if (G <= 4) return launch<float, D, 4>(a, s);
    return launch<float, D, 8>(a, s);
}

}  // namespace

size_t attn_decode_bytes(int D) {
    return kStatusBytes + (size_t)kMaxGrid * (sizeof(int4) + 2 * 16 * (sizeof(float2) + (size_t)D * 4));
}

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s) {
    if (a.bf16) return a.D == 128 ? launch<bf16, 128, 16>(a, s) : launch<bf16, 64, 16>(a, s);
    return a.D == 128 ? launch_f32<128>(a, s) : launch_f32<64>(a, s);
}

cudaError_t launch_attn_short(const AttnArgs& args, const AttnPlan& plan, void* ws, cudaStream_t s) {
    AttnArgs a = args;
    a.ws = ws;
    return a.D == 128 ? launch<bf16, 128, kShortRows, true>(a, s, plan)
                      : launch<bf16, 64, kShortRows, true>(a, s, plan);
}

cudaError_t read_attn_decode_error(int32_t* out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_decode_attn_error, sizeof(int32_t));
    if (e == cudaSuccess && *out != 0) {
        const int32_t zero = 0;
        e = cudaMemcpyToSymbol(g_decode_attn_error, &zero, sizeof(int32_t));
    }
    return e;
}

}  // namespace gdn
