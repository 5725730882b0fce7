// paged.cuh -- where a token of a sequence lives: the index arithmetic that the append and
// attention kernels share.  Plain integer functions, callable on the host too, so that bad
// tables can be checked without a GPU.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {

// A sequence's rows.  New tokens are rows q0 .. q0 + n_q - 1 of the token-major tensors; its
// key-value context is n_kv tokens, of which the new ones are the last n_q, so new token i has
// position past + i with past = n_kv - n_q.  (past < 0: the first -past new tokens precede the
// context; they have no position and attend to nothing.)
struct SeqRows {
    int q0, n_q, n_kv;
    int bad;      // 0, or what is wrong with the tables (1: cu, 3: kv_lens, the GDN_DEVERR codes);
                  // such a sequence is skipped
};

// cu null: n_q_dense tokens per sequence.  kv_lens null: the context is the new tokens.
// The entries are data: every value is checked before anything is addressed with it.
GDN_HD SeqRows seq_rows(const int32_t* cu, const int32_t* kv_lens, int n, int64_t n_q_dense, int64_t n_tokens,
                        int64_t max_kv) {
    SeqRows r;
    int64_t a = (int64_t)n * n_q_dense, b = a + n_q_dense;
    if (cu) {
        a = cu[n];
        b = cu[n + 1];
    }
    const int64_t kv = kv_lens ? kv_lens[n] : b - a;
    const bool cu_ok = a >= 0 && b >= a && b <= n_tokens && (n > 0 || a == 0);
    r.bad = !cu_ok ? 1 : (kv_lens && (kv < 0 || kv > max_kv)) ? 3 : 0;
    r.q0 = r.bad ? 0 : (int)a;
    r.n_q = r.bad ? 0 : (int)(b - a);
    r.n_kv = r.bad ? 0 : (int)kv;
    return r;
}

// Row of the cache (page * page_size + offset) that holds position `pos` of a sequence whose
// table row is `table`, or -1 if the table names a page that does not exist.
GDN_HD int64_t cache_row(const int32_t* table, int64_t pos, int page_shift, int n_pages) {
    const int page = table[pos >> page_shift];
    if (page < 0 || page >= n_pages) return -1;
    return ((int64_t)page << page_shift) + (pos & (((int64_t)1 << page_shift) - 1));
}

}  // namespace gdn
