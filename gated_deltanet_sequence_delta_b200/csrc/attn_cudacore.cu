// attn_cudacore.cu -- causal grouped attention on the CUDA cores, for packed prompts and for
// the paged cache: the fp32 mode of the prompt calls (no TF32), and the careful second pass
// over bf16 tiles whose tensor-core result is not finite.
//
//   o_i = sum_{j <= p_i} e^{s_ij - m_i} v_j / sum_{j <= p_i} e^{s_ij - m_i},  s_ij = scale q_i.k_j,
// p_i the position of row i, in one pass over the keys with the running maximum m and sum.
//
// The rows of a tile are (token, query head of the group) pairs of one key-value head, so the
// group shares each key and value that is staged.  64 rows x 64 keys a step, 256 threads, a
// 4 x 4 block of scores and 4 x D/16 outputs each; row statistics stay within a half-warp.
// Bound: shared-memory reads (8 16-byte reads per 64 FMAs): 0.71 of their rate, half of the fp32 one.
// Measured, fp32: 37.4 TFLOP/s for 8000 tokens (16 heads over 4 of 128), 34.5 of 64; 23 (163 us) for
// 3 x 1111 (8 over 2 of 64).  Where tiles are few, several blocks share a tile's steps and a second kernel
// joins their pieces.
//
// Masked places never enter a sum, neither their scores nor 0 * v_j, so infinities and NaN in
// values a row does not see leave it alone.
#include "attn_common.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

__device__ int g_cc_error;

constexpr int kThreads = 256;
constexpr int kM = 64, kN = 64;
constexpr int kPStride = kN + 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Smem {
    float q[kM][D];
    union {                 // the probabilities take the keys' place once the scores are formed,
        float k[kN][D + 4]; // so that two blocks fit an SM
        float p[kM][kPStride];
    };
    float v[kN][D];
    int64_t row[kN];        // row of k, v that holds each key of the step, -1: none
    int lim[kM];            // last key position each row sees, -1: none
};

template <typename IO>
__device__ __forceinline__ float4 load4(const IO* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&r.x);
    const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&r.y);
    return make_float4(__low2float(a), __high2float(a), __low2float(b), __high2float(b));
}

// A tile's steps may be shared by several blocks, its pieces, `most` of them at most.
struct Piece {
    int index, most;
    float2* ml;           // [most][64] (maximum, sum), and
    float* o;             // [most][64][D] the sums as they are, where there are two pieces or more
};
// With few tiles (most at its limit) the longest tile's chain of steps is the time: pieces from three
// steps on.  With more, blocks share the SMs, and a piece has to be worth its way through memory: tiles
// of six steps or more, two a piece (16 x 200 tokens, 8 heads over 2 of 64, tiles of four steps: 43 us
// whole, 56 in two pieces).  All of this is measured on prompts of up to 1111 tokens.  Over a long past four
// pieces a tile leave most of the device idle: 4 tokens over 30K, 8 heads over 2 of 128, take 1.30 ms for 61 MB.
constexpr int kMostPieces = 4;
__host__ __device__ constexpr int split_steps(int most) { return most == kMostPieces ? 3 : 6; }
__device__ __forceinline__ int pieces_of(int keys, int most) {
    const int steps = (keys + kN - 1) / kN;
    if (steps < split_steps(most)) return 1;
    return min(most, most == kMostPieces ? steps : steps / 2);
}
// Keys that a tile's last row sees.
__device__ __forceinline__ int tile_keys(const SeqRows& sq, int64_t row0, int per, int64_t row_end) {
    return max(sq.n_kv - sq.n_q + (int)((min(row0 + kM, row_end) - 1) / per) + 1, 0);
}

// One tile: rows row0 .. row0 + 63 of sequence n's (token, head) rows, row r being token
// r / per and query head head0 + r % per, against key-value head kvh.
template <typename IO, int D>
__device__ void attn_tile(const AttnArgs& a, Smem<D>& sm, const SeqRows& sq, int n, int kvh, int64_t row0, int per,
                          int head0, int64_t row_end, Piece piece) {
    const int keys = tile_keys(sq, row0, per, row_end), steps = (keys + kN - 1) / kN;
    const int pieces = pieces_of(keys, piece.most);
    if (piece.index >= pieces) return;
    const int begin = (int)((int64_t)steps * piece.index / pieces) * kN;
    const int end = (int)min((int64_t)steps * (piece.index + 1) / pieces * kN, (int64_t)keys);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int past = sq.n_kv - sq.n_q;
    const IO* q = (const IO*)a.q;
    const IO* K = (const IO*)a.kv.k;
    const IO* V = (const IO*)a.kv.v;
    __syncthreads();                 // the previous tile's reads of shared memory are over
    for (int i = tid; i < kM; i += kThreads) {
        const int64_t r = row0 + i;
        sm.lim[i] = r < row_end ? past + (int)(r / per) : -1;
    }
    {
        constexpr int NL = kM * (D / 4) / kThreads, kRowsAt = kThreads / (D / 4);
        const int r0 = tid / (D / 4), c = (tid % (D / 4)) * 4;
        float4 x[NL];
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int64_t r = row0 + r0 + i * kRowsAt;
            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < row_end) x[i] = load4(q + ((sq.q0 + r / per) * a.HQ + head0 + (int)(r % per)) * D + c);
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) *reinterpret_cast<float4*>(&sm.q[r0 + i * kRowsAt][c]) = x[i];
    }
    __syncthreads();
    int lim[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) lim[i] = sm.lim[ty * 4 + i];
    const int lim_lo = row0 + kM <= row_end ? past + (int)(row0 / per) : -1;
    const float sc = a.scale * kLog2e;

    float o[4][D / 16], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
    }
    for (int j0 = begin; j0 < end; j0 += kN) {
        if (tid < kN) {
            int64_t row = -1;
            const int pos = j0 + tid;
            if (pos < end) {
                if (a.kv.table) {
                    row = cache_row(a.kv.table + (int64_t)n * a.kv.max_pages, pos, a.kv.page_shift, a.kv.n_pages);
                    if (row < 0) atomicMax(&g_cc_error, GDN_DEVERR_PAGE);
                } else {
                    row = sq.q0 + pos;
                }
            }
            sm.row[tid] = row;
        }
        __syncthreads();
        // four rows of a thread's keys and values in flight before the first is stored (eight at once
        // would cost the second block of an SM at D = 128)
        constexpr int kRowsAt = kThreads / (D / 4);
        const int lr = tid / (D / 4), lc = (tid % (D / 4)) * 4;
#pragma unroll 1
        for (int b = 0; b < kN; b += 4 * kRowsAt) {
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = sm.row[b + lr + i * kRowsAt];
                x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row >= 0) {
                    const int64_t at = (row * a.HKV + kvh) * D + lc;
                    x[i] = load4(K + at);
                    y[i] = load4(V + at);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                *reinterpret_cast<float4*>(&sm.k[b + lr + i * kRowsAt][lc]) = x[i];
                *reinterpret_cast<float4*>(&sm.v[b + lr + i * kRowsAt][lc]) = y[i];
            }
        }
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 qa[4], kb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qa[i] = *reinterpret_cast<const float4*>(&sm.q[ty * 4 + i][d]);
#pragma unroll
            for (int j = 0; j < 4; ++j) kb[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][d]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(qa[i].x, kb[j].x, s[i][j]);
                    s[i][j] = fmaf(qa[i].y, kb[j].y, s[i][j]);
                    s[i][j] = fmaf(qa[i].z, kb[j].z, s[i][j]);
                    s[i][j] = fmaf(qa[i].w, kb[j].w, s[i][j]);
                }
        }
        __syncthreads();             // every score is formed: p may overwrite k
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = j0 + tx + 16 * j <= lim[i] ? s[i][j] * sc : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float base = mx == -INFINITY ? 0.f : mx;      // a row that has seen no key yet
            const float alpha = exp2f(m[i] - base);
            m[i] = mx;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = j0 + tx + 16 * j <= lim[i] ? exp2f(s[i][j] - base) : 0.f;
                sm.p[ty * 4 + i][tx + 16 * j] = p;
                sum += p;
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l[i] = l[i] * alpha + sum;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= alpha;
        }
        __syncwarp();                // a row's p is written and read by the same half-warp
        if (j0 + kN - 1 <= lim_lo) {
#pragma unroll 2
            for (int j = 0; j < kN; j += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(&sm.p[ty * 4 + i][j]);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const float4 v = *reinterpret_cast<const float4*>(&sm.v[j + jj][c * 64 + tx * 4]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float pi = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
                            o[i][c * 4 + 0] = fmaf(pi, v.x, o[i][c * 4 + 0]);
                            o[i][c * 4 + 1] = fmaf(pi, v.y, o[i][c * 4 + 1]);
                            o[i][c * 4 + 2] = fmaf(pi, v.z, o[i][c * 4 + 2]);
                            o[i][c * 4 + 3] = fmaf(pi, v.w, o[i][c * 4 + 3]);
                        }
                    }
            }
        } else {                     // some row does not see every key of this step
            const int stop = min(kN, end - j0);
            for (int j = 0; j < stop; ++j) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(&sm.v[j][c * 64 + tx * 4]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (j0 + j <= lim[i]) {
                            const float pi = sm.p[ty * 4 + i][j];
                            o[i][c * 4 + 0] = fmaf(pi, v.x, o[i][c * 4 + 0]);
                            o[i][c * 4 + 1] = fmaf(pi, v.y, o[i][c * 4 + 1]);
                            o[i][c * 4 + 2] = fmaf(pi, v.z, o[i][c * 4 + 2]);
                            o[i][c * 4 + 3] = fmaf(pi, v.w, o[i][c * 4 + 3]);
                        }
                }
            }
        }
        __syncthreads();             // before the next step overwrites k, v
    }
    if (pieces > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = piece.index * kM + ty * 4 + i;
            if (row0 + ty * 4 + i >= row_end) continue;
            if (tx == 0) piece.ml[r] = make_float2(m[i], l[i]);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                *reinterpret_cast<float4*>(piece.o + (int64_t)r * D + c * 64 + tx * 4) =
                    make_float4(o[i][c * 4], o[i][c * 4 + 1], o[i][c * 4 + 2], o[i][c * 4 + 3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = row0 + ty * 4 + i;
        if (r >= row_end) continue;
        const int64_t at = ((sq.q0 + r / per) * a.HQ + head0 + (int)(r % per)) * D;
        const bool empty = lim[i] < 0;                 // no key: zero
        const float inv = empty ? 0.f : 1.0f / l[i];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            const int64_t e = at + (c >> 2) * 64 + tx * 4 + (c & 3);
            float x = empty ? 0.f : o[i][c] * inv;
            if (a.z && !empty) x = gate_out(x, load_elem((const IO*)a.z, e));
            store_elem((IO*)a.o, e, x);
        }
    }
}

// Where the pieces of a (tile, key-value head) are kept: behind the plan.
struct Pieces {
    float2* ml;
    float* o;
    int most;
    __device__ __forceinline__ Piece of(int64_t tile_head, int index, int D) const {
        return Piece{index, most, ml + tile_head * most * kM, o + tile_head * most * kM * D};
    }
};

// Block (tile * most + piece, key-value head): long tiles come first, a tile's pieces side by side.
template <typename IO, int D>
__global__ void __launch_bounds__(kThreads, 2) attn_cc_kernel(AttnArgs a, AttnPlan plan, Pieces pieces) {
    extern __shared__ float4 smem_raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
    tc::grid_dependency_sync();
    const int tile = blockIdx.x / pieces.most, index = blockIdx.x - tile * pieces.most;
    if (tile >= plan.counts[0]) return;
    const PlanTile it = plan.tiles[tile];
    const SeqRows sq = {it.q0, it.n_q, it.n_kv, 0};
    const int G = a.HQ / a.HKV;
    attn_tile<IO, D>(a, sm, sq, it.n, blockIdx.y, (int64_t)it.index * kM, G, blockIdx.y * G, (int64_t)sq.n_q * G,
                     pieces.of((int64_t)tile * a.HKV + blockIdx.y, index, D));
}

// Joins a tile's pieces, in order.  A thread four columns of a row.
template <typename IO, int D>
__global__ void __launch_bounds__(kThreads) attn_cc_join_kernel(AttnArgs a, AttnPlan plan, Pieces pieces) {
    tc::grid_dependency_sync();
    const int tile = blockIdx.x, kvh = blockIdx.y, G = a.HQ / a.HKV;
    if (tile >= plan.counts[0]) return;
    const PlanTile it = plan.tiles[tile];
    const SeqRows sq = {it.q0, it.n_q, it.n_kv, 0};
    const int64_t row0 = (int64_t)it.index * kM, row_end = (int64_t)sq.n_q * G;
    const int n = pieces_of(tile_keys(sq, row0, G, row_end), pieces.most);
    if (n == 1) return;
    const Piece p = pieces.of((int64_t)tile * a.HKV + kvh, 0, D);
    for (int u = threadIdx.x; u < kM * (D / 4); u += kThreads) {
        const int row = u / (D / 4), c = (u % (D / 4)) * 4;
        const int64_t r = row0 + row;
        if (r >= row_end) break;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < n; ++k) m = fmaxf(m, p.ml[k * kM + row].x);
        const float base = m == -INFINITY ? 0.f : m;
        for (int k = 0; k < n; ++k) {
            const float2 ml = p.ml[k * kM + row];
            // (a row that sees no key of the piece has m = -inf and zeros there)
            const float f = exp2f(ml.x - base);
            const float4 y = *reinterpret_cast<const float4*>(p.o + (int64_t)(k * kM + row) * D + c);
            l = fmaf(f, ml.y, l);
            o.x = fmaf(f, y.x, o.x);
            o.y = fmaf(f, y.y, o.y);
            o.z = fmaf(f, y.z, o.z);
            o.w = fmaf(f, y.w, o.w);
        }
        const bool empty = sq.n_kv - sq.n_q + (int)(r / G) < 0;          // no key: zero
        const float inv = empty ? 0.f : 1.0f / l, x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
        const int64_t at = ((sq.q0 + r / G) * a.HQ + kvh * G + (int)(r % G)) * D + c;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y = empty ? 0.f : x[e];
            if (a.z && !empty) y = gate_out(y, load_elem((const IO*)a.z, at + e));
            store_elem((IO*)a.o, at + e, y);
        }
    }
}

// The rows that the tensor-core kernel listed.
template <int D>
__global__ void __launch_bounds__(kThreads, 2) attn_redo_kernel(AttnArgs a, AttnPlan plan) {
    extern __shared__ float4 smem_raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
    tc::grid_dependency_sync();
    const int G = a.HQ / a.HKV, count = min(plan.counts[1], plan.max_redo);
    for (int i = blockIdx.x; i < count; i += gridDim.x) {
        const int4 it = plan.redo[i];
        const SeqRows sq = seq_rows(a, it.x);
        const int64_t end = min((int64_t)it.z + it.w, (int64_t)sq.n_q * G);
        if (it.z < end) attn_tile<__nv_bfloat16, D>(a, sm, sq, it.x, it.y, it.z, G, it.y * G, end,
                                                      Piece{0, 1, nullptr, nullptr});
    }
}

// How many pieces a tile may have: enough that a call's blocks fill the device twice over, since a block
// alone takes 6 us a step, one after the other, and two or three on an SM 4.6 us a step.  In pieces against
// whole, fp32: 70 / 119 us (1111 tokens, 8 heads over 2 of 64), 35 / 56 (500), 71 / 129 (700, 4 over 1 of
// 128), 164 / 171 (3 x 1111); 190 tokens, 8 over 8 of 128: 45 / 42.
constexpr int kBlocks = 888;
int most_pieces(const AttnPlan& plan, int HKV) {
    const int64_t tiles = (int64_t)plan.max_tiles * HKV;
    return (int)max((int64_t)1, min((int64_t)kMostPieces, (kBlocks + tiles - 1) / max(tiles, (int64_t)1)));
}
Pieces pieces_at(void* ws, const AttnPlan& plan, int HKV, int D, size_t* bytes) {
    const int most = most_pieces(plan, HKV);
    const size_t at = (plan.bytes + 255) / 256 * 256, rows = most > 1 ? (size_t)plan.max_tiles * HKV * most * kM : 0;
    uint8_t* b = static_cast<uint8_t*>(ws) + at;
    *bytes = at + rows * (D * sizeof(float) + sizeof(float2));
    return Pieces{reinterpret_cast<float2*>(b + rows * D * sizeof(float)), reinterpret_cast<float*>(b), most};
}

template <typename IO, int D>
cudaError_t launch_cc(const AttnArgs& a, const AttnPlan& plan, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem((const void*)attn_cc_kernel<IO, D>, sizeof(Smem<D>), done);
    if (e != cudaSuccess) return e;
    size_t bytes;
    Pieces pieces = pieces_at(a.ws, plan, a.HKV, D, &bytes);
    // (the longest context that there can be)
    const int64_t longest = a.kv.table ? (int64_t)a.kv.max_pages << a.kv.page_shift : a.cu ? a.n_tokens : a.T;
    if (longest <= (split_steps(pieces.most) - 1) * kN) pieces.most = 1;
    e = launch_pdl(attn_cc_kernel<IO, D>, dim3((unsigned)(plan.max_tiles * pieces.most), (unsigned)a.HKV),
                   dim3(kThreads), sizeof(Smem<D>), s, a, plan, pieces);
    if (e != cudaSuccess) return e;
    count_launch();
    if (pieces.most == 1) return cudaSuccess;
    e = launch_pdl(attn_cc_join_kernel<IO, D>, dim3((unsigned)plan.max_tiles, (unsigned)a.HKV), dim3(kThreads), 0, s, a,
                   plan, pieces);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace

cudaError_t launch_attn_redo(const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
    const size_t smem = a.D == 128 ? sizeof(Smem<128>) : sizeof(Smem<64>);
    const auto f = a.D == 128 ? attn_redo_kernel<128> : attn_redo_kernel<64>;
    static std::atomic<uint64_t> done[2];
    cudaError_t e = allow_smem((const void*)f, smem, done[a.D == 128]);
    if (e != cudaSuccess) return e;
    // the list is empty unless something is not finite: a grid that starts and ends in about the
    // launch's own time, and still spreads a list over the device
    e = launch_pdl(f, dim3(148), dim3(kThreads), smem, s, a, p);
    if (e == cudaSuccess) count_launch();
    return e;
}

size_t attn_cudacore_bytes(int64_t n_tokens, int n_seqs, int HQ, int HKV, int D) {
    size_t bytes;
    pieces_at(nullptr, attn_plan(nullptr, n_tokens, n_seqs, 0, HQ / HKV, kM, 0, 0), HKV, D, &bytes);
    return bytes;
}

cudaError_t launch_attn_cudacore(const AttnArgs& a, cudaStream_t s) {
    if (a.n_tokens == 0 || a.n_seqs == 0) return cudaSuccess;
    const int G = a.HQ / a.HKV;
    const AttnPlan plan = attn_plan(a.ws, a.n_tokens, a.n_seqs, 0, G, kM, 0, 0);
    cudaError_t e = launch_attn_plan(a, plan, G, kM, 0, s);
    if (e != cudaSuccess) return e;
    if (a.bf16)
        return a.D == 128 ? launch_cc<__nv_bfloat16, 128>(a, plan, s) : launch_cc<__nv_bfloat16, 64>(a, plan, s);
    return a.D == 128 ? launch_cc<float, 128>(a, plan, s) : launch_cc<float, 64>(a, plan, s);
}

cudaError_t read_attn_cudacore_error(int32_t* out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_cc_error, sizeof(int32_t));
    if (e == cudaSuccess && *out != 0) {
        const int32_t zero = 0;
        e = cudaMemcpyToSymbol(g_cc_error, &zero, sizeof(int32_t));
    }
    return e;
}

}  // namespace gdn
