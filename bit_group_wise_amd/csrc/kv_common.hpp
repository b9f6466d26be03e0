// kv_common.hpp -- device-side definitions shared by the key/value cache
// kernels: where a token's row lies, and how its groups decode.
#pragma once

#include "q4_common.hpp"
#include "q4_internal.hpp"

namespace q4 {

// q4_kv_cache / q4_kv_batch as the kernels take them (validated).
struct KvHalf {  // keys or values
    uint8_t *codes;
    void *scales;
    uint8_t *zeros;
};
struct KvCache {
    KvHalf k, v;
    int pages, page_shift, heads, dim, g;
};
struct KvBatch {
    const int32_t *table;
    const int32_t *lens;
    const int32_t *starts;
    int64_t tokens;
    int table_width, seqs, max_new, max_len;
};

inline KvCache kv_cache_args(const q4_kv_cache &c)
{
    return KvCache{{c.k_codes, c.k_scales, c.k_zeros},
                   {c.v_codes, c.v_scales, c.v_zeros},
                   (int)c.pages, __builtin_ctz((unsigned)c.page), c.heads, c.dim, c.g};
}
inline KvBatch kv_batch_args(const q4_kv_batch &b)
{
    return KvBatch{b.table, b.lens, b.starts, b.tokens, b.table_width, b.seqs, b.max_new, b.max_len};
}

// One sequence's share of a batch: its cached length, the packed row of its
// first new token and their number.  Values that do not fit the caller's
// bounds are cut to them, so that no index derived from them leaves an array.
struct KvSeq {
    int len, first, fresh;
};
__device__ __forceinline__ KvSeq kv_seq(const KvBatch &b, int seq)
{
    KvSeq s;
    s.len = min(max(b.lens[seq], 0), b.max_len);
    if (b.starts) {
        const int64_t s0 = min((int64_t)max(b.starts[seq], 0), b.tokens);
        const int64_t s1 = min((int64_t)max(b.starts[seq + 1], 0), b.tokens);
        s.first = (int)s0;
        s.fresh = (int)min(max(s1 - s0, (int64_t)0), (int64_t)b.max_new);
    } else {
        s.first = seq;
        s.fresh = 1;
    }
    return s;
}

// Row (over the pool's [pages, heads, page]) of token t of a sequence in head
// h, or -1 where the table names no page of the pool.  t is in [0, max_len).
__device__ __forceinline__ int64_t kv_row(const KvCache &c, const int32_t *table_row, int t, int h)
{
    const int p = table_row[t >> c.page_shift];
    if ((unsigned)p >= (unsigned)c.pages)
        return -1;
    return (((int64_t)p * c.heads + h) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
}

// Bytes of zero-points a row (INT4-asym): two groups a byte.
__host__ __device__ constexpr int kv_zero_bytes(int dim, int g) { return (dim / g + 1) / 2; }

// Scale of group j of a row, and (asym) its zero-point.
template <int FMT>
__device__ __forceinline__ float kv_scale(const KvHalf &x, int64_t row, int groups, int j)
{
    if constexpr (f32_absmax(FMT))
        return ((const float *)x.scales)[row * groups + j];
    else
        return (float)((const _Float16 *)x.scales)[row * groups + j];
}
template <int FMT>
__device__ __forceinline__ float kv_zero(const KvHalf &x, int64_t row, int groups, int j)
{
    if constexpr (FMT == Q4_INT4_ASYM)
        return (float)((x.zeros[row * ((groups + 1) / 2) + (j >> 1)] >> (4 * (j & 1))) & 15);
    else
        return FMT == Q4_INT4_SYM ? 8.0f : 0.0f;
}
// Calls fn(integral_constant<FMT>) for the run-time format.
template <int V>
struct KvInt {
    static constexpr int value = V;
};
template <class F>
hipError_t kv_by_format(int f, F &&fn)
{
    switch (f) {
    case Q4_NF4: return fn(KvInt<Q4_NF4>{});
    case Q4_INT4_SYM: return fn(KvInt<Q4_INT4_SYM>{});
    case Q4_INT4_ASYM: return fn(KvInt<Q4_INT4_ASYM>{});
    case Q4_FP4: return fn(KvInt<Q4_FP4>{});
    }
    return hipErrorInvalidValue;
}

hipError_t launch_kv_append(int f, const KvCache &c, const KvBatch &b, int in_t, const void *k,
                            int64_t kts, int64_t khs, const void *v, int64_t vts, int64_t vhs,
                            hipStream_t s);
hipError_t launch_kv_read(int f, const KvCache &c, const KvBatch &b, int out_t, void *k, void *v,
                          hipStream_t s);
size_t kv_attention_workspace(const KvCache &c, const KvBatch &b, int q_heads, int window, bool mass);
hipError_t launch_kv_attention(int f, const KvCache &c, const KvBatch &b, int act_t, const void *q,
                               int64_t qts, int64_t qhs, int q_heads, float scale, int window,
                               void *out, float *lse, float *mass, int64_t mass_width,
                               void *workspace, hipStream_t s);
hipError_t launch_kv_evict(int f, const KvCache &c, const KvBatch &b, const float *mass,
                           int64_t mass_width, const int32_t *new_table, int new_table_width,
                           int budget, int recent, int32_t *new_lens, float *new_mass,
                           int64_t new_width, int32_t *kept, hipStream_t s);

}  // namespace q4
