// attn_append.cu -- new tokens enter the paged key-value cache: queries and keys are rotated by
// their positions, keys and values are written to the pages, the rotated queries returned.
//
// Rotation.  Pair i of a head (elements i and i + R/2, or 2i and 2i + 1) turns by the angle
// pos * inv_freq[i]:  (a, b) -> (a cos - b sin, b cos + a sin).  A float product would lose the
// angle of far positions (at 2^18 its last bit is 2^-6 rad), so the angle is formed in turns in
// double, pos * inv_freq / (2 pi), and only its fraction, in [-1/2, 1/2], goes to sincospif: the
// error at position p stays below p * inv_freq * 2^-53 turns plus float's own rounding.
//
// Bound: HBM (every element is read once and written once).  One block takes a few tokens; it
// forms their rotary/2 sines and cosines once (the heads share them) in shared memory and then
// walks (token, head, pair of 16-byte chunks) units.  A unit holds both halves of its pairs, so
// every access is 16 bytes wide and in-place rotation of q is safe.
//
// Measured: 37K tokens of 32 + 2 x 8 heads of 128, bf16, from the fused projection: 162.5 us for 908 MB
// (5.6 TB/s, 0.87 of a copy); 64 tokens: 3.4 us, one chain of loads.
#include "attn_common.cuh"

namespace gdn {
namespace {

__device__ int g_append_error;

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;          // tokens per block

template <typename IO>
struct Chunk {                      // 16 bytes of a head
    static constexpr int N = 16 / sizeof(IO);
    float x[N];
    __device__ __forceinline__ void load(const IO* p) {
        const uint4 r = *reinterpret_cast<const uint4*>(p);
        const IO* e = reinterpret_cast<const IO*>(&r);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = load_elem(e, i);
    }
    __device__ __forceinline__ void store(IO* p) const {
        uint4 r;
        IO* e = reinterpret_cast<IO*>(&r);
#pragma unroll
        for (int i = 0; i < N; ++i) store_elem(e, i, x[i]);
        *reinterpret_cast<uint4*>(p) = r;
    }
};

template <typename IO>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a, int tok_per_block, int unit_blocks) {
    constexpr int N = Chunk<IO>::N;
    __shared__ float2 s_cs[kMaxTok][64];        // (cos, sin) of each token's pairs
    __shared__ int s_seq[kMaxTok];
    __shared__ int64_t s_row[kMaxTok];          // cache row, -1: not written
    __shared__ int s_pos[kMaxTok];              // position, negative: the token is skipped
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * tok_per_block;
    const int nt = (int)min((int64_t)tok_per_block, a.n_tokens - t0);
    if (tid < kMaxTok) s_seq[tid] = -1;
    __syncthreads();
    // which sequence each token belongs to: every thread looks at its share of the table
    if (a.cu) {
        for (int n = tid; n < a.n_seqs; n += kThreads) {
            const int64_t lo = a.cu[n], hi = a.cu[n + 1];
            for (int i = 0; i < nt; ++i)
                if (lo <= t0 + i && t0 + i < hi) s_seq[i] = n;
            if (blockIdx.x == 0 && (lo < 0 || hi < lo || hi > a.n_tokens || (n == 0 && lo != 0)))
                atomicMax(&g_append_error, GDN_DEVERR_CU_SEQLENS);
        }
    } else if (tid < nt) {
        s_seq[tid] = (int)(t0 + tid);           // one token per sequence
    }
    __syncthreads();
    if (tid < nt) {
        const int n = s_seq[tid];
        int pos = -1;
        int64_t row = -1;
        if (n >= 0) {
            const SeqRows r = seq_rows(a.cu, a.kv_lens, n, 1, a.n_tokens, (int64_t)a.max_pages << a.page_shift);
            if (!r.bad) {
                pos = r.n_kv - r.n_q + (int)(t0 + tid - r.q0);
                if (pos >= 0) {
                    row = cache_row(a.table + (int64_t)n * a.max_pages, pos, a.page_shift, a.n_pages);
                    if (row < 0) atomicMax(&g_append_error, GDN_DEVERR_PAGE);
                }
            } else {
                atomicMax(&g_append_error, r.bad);
            }
        }
        s_pos[tid] = pos;
        s_row[tid] = row;
    }
    __syncthreads();
    const int half = a.rotary / 2;
    for (int i = tid; i < nt * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        if (s_pos[t] >= 0) {
            const double turns = (double)s_pos[t] * (double)a.inv_freq[p] * 0.15915494309189535;
            float sn, cs;
            sincospif((float)(turns - rint(turns)) * 2.0f, &sn, &cs);
            s_cs[t][p] = make_float2(cs, sn);
        }
    }
    __syncthreads();

    const int heads = (a.q ? a.HQ : 0) + 2 * a.HKV;
    const int upd = a.D / (2 * N);              // units per head: a power of two, 4 to 16
    // a thread keeps its unit of a head and steps through the (token, head) pairs
    const int u0 = blockIdx.y * kThreads + tid, c = u0 % upd, step = kThreads * unit_blocks / upd;
    int t = u0 / upd / heads, th = u0 / upd - t * heads;
#pragma unroll 2
    for (; t < nt; th += step) {
        while (th >= heads) {
            th -= heads;
            ++t;
        }
        if (t >= nt) break;
        int h = th;
        if (s_pos[t] < 0) continue;
        const int64_t tok = t0 + t;
        const IO* src;
        IO* dst;
        bool turn = true;
        if (a.q && h < a.HQ) {
            src = (const IO*)a.q + tok * a.q_stride + (int64_t)h * a.D;
            dst = (IO*)a.q_out + (tok * a.HQ + h) * a.D;
        } else {
            if (a.q) h -= a.HQ;
            if (s_row[t] < 0) continue;
            const bool is_v = h >= a.HKV;
            if (is_v) h -= a.HKV;
            src = is_v ? (const IO*)a.v + tok * a.v_stride : (const IO*)a.k + tok * a.k_stride;
            src += (int64_t)h * a.D;
            dst = (IO*)(is_v ? a.v_cache : a.k_cache) + (s_row[t] * a.HKV + h) * a.D;
            turn = !is_v;
        }
        // the unit's two chunks: the two halves of N pairs where the layout splits them, else
        // 2 N neighbours
        const int rot_units = half / N;
        int e0 = 2 * N * c, e1 = e0 + N;
        const bool rot = turn && c < rot_units;
        if (rot && !a.interleaved) {
            e0 = N * c;
            e1 = e0 + half;
        }
        Chunk<IO> x, y;
        x.load(src + e0);
        y.load(src + e1);
        if (rot) {
            const float2* cs = s_cs[t] + N * c;
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    const float2 w0 = cs[i], w1 = cs[N / 2 + i];
                    const float x0 = x.x[2 * i], x1 = x.x[2 * i + 1], y0 = y.x[2 * i], y1 = y.x[2 * i + 1];
                    x.x[2 * i] = x0 * w0.x - x1 * w0.y;
                    x.x[2 * i + 1] = x1 * w0.x + x0 * w0.y;
                    y.x[2 * i] = y0 * w1.x - y1 * w1.y;
                    y.x[2 * i + 1] = y1 * w1.x + y0 * w1.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float2 w = cs[i];
                    const float x0 = x.x[i], y0 = y.x[i];
                    x.x[i] = x0 * w.x - y0 * w.y;
                    y.x[i] = y0 * w.x + x0 * w.y;
                }
            }
        }
        x.store(dst + e0);
        y.store(dst + e1);
    }
}

}  // namespace

cudaError_t launch_attn_append(const AppendArgs& a, cudaStream_t s) {
    if (a.n_tokens == 0 || a.n_seqs == 0) return cudaSuccess;
    const int n = a.bf16 ? 8 : 4;
    const int units = ((a.q ? a.HQ : 0) + 2 * a.HKV) * (a.D / (2 * n));     // per token
    // Few tokens: one per block and its units over several blocks, one unit a thread, since the
    // call's time is then the latency of one chain of loads.  Many: kMaxTok tokens share a block and
    // their sines.  Few against many, bf16, 16 + 2 x 4 heads of 128: 3.3 / 6.7 us at 64 tokens, 6.7 / 7.0
    // at 1024, 10.2 / 8.7 at 2048, 17.9 / 12.3 at 4096.
    const bool few = a.n_tokens < 1024;
    const int tok = few ? 1 : kMaxTok;
    const int ub = few ? (units + kThreads - 1) / kThreads : 1;
    const dim3 grid((unsigned)((a.n_tokens + tok - 1) / tok), (unsigned)ub);
    if (a.bf16)
        append_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a, tok, ub);
    else
        append_kernel<float><<<grid, kThreads, 0, s>>>(a, tok, ub);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch();
    return e;
}

cudaError_t read_append_error(int32_t* out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_append_error, sizeof(int32_t));
    if (e == cudaSuccess && *out != 0) {
        const int32_t zero = 0;
        e = cudaMemcpyToSymbol(g_append_error, &zero, sizeof(int32_t));
    }
    return e;
}

}  // namespace gdn
