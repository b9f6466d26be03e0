// kv_attn.hip -- attention over the 4-bit key/value cache (q4_kv_attention).
//
// Mathematics: x_t = scale <q, K_t> over the tokens a row sees, out = sum_t
// softmax(x)_t V_t, in one pass with the running maximum m and sum l of the
// softmax: a tile of tokens with scores x raises m to m', and sums and output
// so far are scaled by exp(m - m').  The mass of a token, the sum of the
// softmax weights that all rows put on it, needs the final statistics and is
// a second pass over the scores, one thread a token, in a fixed order.
//
// One workgroup per (new token, query head) here, one thread per cached token
// for the scores and per value for the output.
#include "kv_common.hpp"

namespace q4 {
namespace {

constexpr int kBlock = 256;

__constant__ float c_nf4[16] = {kNF4[0], kNF4[1], kNF4[2],  kNF4[3],  kNF4[4],  kNF4[5],
                                kNF4[6], kNF4[7], kNF4[8],  kNF4[9],  kNF4[10], kNF4[11],
                                kNF4[12], kNF4[13], kNF4[14], kNF4[15]};
__constant__ float c_fp4[16] = {kFP4[0], kFP4[1], kFP4[2],  kFP4[3],  kFP4[4],  kFP4[5],
                                kFP4[6], kFP4[7], kFP4[8],  kFP4[9],  kFP4[10], kFP4[11],
                                kFP4[12], kFP4[13], kFP4[14], kFP4[15]};

__device__ __forceinline__ float act_f32(const uint16_t *p, int act)
{
    return act == Q4_F16 ? h2f(*p) : bf2f(*p);
}

// <q, K_row> with q in LDS as binary32.
template <int FMT>
__device__ float dot_row(const KvHalf &x, int64_t row, const float *q, int dim, int g, const float *tbl)
{
    const int groups = dim / g;
    float s = 0.0f;
    for (int j = 0; j < groups; ++j) {
        const float z = kv_zero<FMT>(x, row, groups, j);
        float a = 0.0f;
        for (int d = j * g; d < j * g + g; d += 8) {
            const uint32_t w = *(const uint32_t *)(x.codes + row * (dim >> 1) + (d >> 1));
            for (int i = 0; i < 8; ++i)
                a = __builtin_fmaf(kv_level<FMT>(w >> (4 * i), tbl) - z, q[d + i], a);
        }
        s = __builtin_fmaf(a, kv_scale<FMT>(x, row, groups, j), s);
    }
    return s;
}

template <int FMT>
__global__ __launch_bounds__(kBlock) void kv_attn_simple(KvCache c, KvBatch b, int act,
                                                         const uint16_t *__restrict__ q, int64_t qts,
                                                         int64_t qhs, int q_heads, float scale,
                                                         int window, uint16_t *__restrict__ out,
                                                         float *__restrict__ lse, float *__restrict__ stat)
{
    __shared__ float tbl[16], qs[256], ps[kBlock], red[kBlock];
    const int seq = blockIdx.z, hq = blockIdx.y, i = blockIdx.x, tid = threadIdx.x;
    const KvSeq s = kv_seq(b, seq);
    if (i >= s.fresh)
        return;
    const int h = hq / (q_heads / c.heads);
    const int64_t tok = s.first + i;
    if (tid < 16)
        tbl[tid] = FMT == Q4_FP4 ? c_fp4[tid] : c_nf4[tid];
    if (tid < c.dim)
        qs[tid] = act_f32(q + tok * qts + hq * qhs + tid, act);
    __syncthreads();
    const int32_t *table = b.table + (int64_t)seq * b.table_width;
    const int pos = s.len - s.fresh + i;
    const int t0 = window > 0 ? max(0, pos - window + 1) : 0;
    float m = -__builtin_inff(), l = 0.0f, o = 0.0f;
    for (int t = t0; t <= pos; t += kBlock) {
        const int64_t row = t + tid <= pos ? kv_row(c, table, t + tid, h) : -1;
        const float x = row < 0 ? -__builtin_inff() : scale * dot_row<FMT>(c.k, row, qs, c.dim, c.g, tbl);
        red[tid] = x;
        __syncthreads();
        for (int d = kBlock / 2; d; d >>= 1) {
            if (tid < d)
                red[tid] = fmaxf(red[tid], red[tid + d]);
            __syncthreads();
        }
        const float mn = fmaxf(m, red[0]);
        __syncthreads();
        const float p = row < 0 ? 0.0f : __expf(x - mn);
        ps[tid] = red[tid] = p;
        __syncthreads();
        for (int d = kBlock / 2; d; d >>= 1) {
            if (tid < d)
                red[tid] += red[tid + d];
            __syncthreads();
        }
        const float f = m == -__builtin_inff() ? 0.0f : __expf(m - mn);
        l = l * f + red[0];
        m = mn;
        if (tid < c.dim) {
            o *= f;
            for (int u = 0; u < kBlock && t + u <= pos; ++u) {
                const int64_t r = kv_row(c, table, t + u, h);
                if (r < 0)
                    continue;
                const int groups = c.dim / c.g, j = tid / c.g;
                const uint32_t code = c.v.codes[r * (c.dim >> 1) + (tid >> 1)] >> (4 * (tid & 1));
                const float val = (kv_level<FMT>(code, tbl) - kv_zero<FMT>(c.v, r, groups, j)) *
                                  kv_scale<FMT>(c.v, r, groups, j);
                o = __builtin_fmaf(ps[u], val, o);
            }
        }
        __syncthreads();
    }
    if (tid < c.dim) {
        const float v = l > 0.0f ? o / l : 0.0f;
        out[(tok * q_heads + hq) * c.dim + tid] = (uint16_t)(act == Q4_F16 ? f2h_bits(v) : f2bf_bits(v));
    }
    if (tid == 0) {
        const float v = l > 0.0f ? m + logf(l) : -__builtin_inff();
        if (lse)
            lse[tok * q_heads + hq] = v;
        if (stat)
            stat[tok * q_heads + hq] = v;
    }
}

// mass[b, h, t] += sum over rows of exp(x_t - lse); one thread a token.
template <int FMT>
__global__ __launch_bounds__(kBlock) void kv_mass_simple(KvCache c, KvBatch b, int act,
                                                         const uint16_t *__restrict__ q, int64_t qts,
                                                         int64_t qhs, int q_heads, float scale,
                                                         int window, const float *__restrict__ stat,
                                                         float *__restrict__ mass, int64_t mass_width)
{
    __shared__ float tbl[16], qs[256];
    const int seq = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
    const KvSeq s = kv_seq(b, seq);
    const int t = blockIdx.x * kBlock + tid;
    if ((int)blockIdx.x * kBlock >= s.len)
        return;
    if (tid < 16)
        tbl[tid] = FMT == Q4_FP4 ? c_fp4[tid] : c_nf4[tid];
    const int32_t *table = b.table + (int64_t)seq * b.table_width;
    const int64_t row = t < s.len ? kv_row(c, table, t, h) : -1;
    const int G = q_heads / c.heads;
    float sum = 0.0f;
    for (int r = 0; r < s.fresh * G; ++r) {
        const int i = r / G, hq = h * G + r % G;
        const int64_t tok = s.first + i;
        const int pos = s.len - s.fresh + i;
        __syncthreads();
        if (tid < c.dim)
            qs[tid] = act_f32(q + tok * qts + hq * qhs + tid, act);
        __syncthreads();
        if (row >= 0 && t <= pos && (window <= 0 || t > pos - window))
            sum += __expf(scale * dot_row<FMT>(c.k, row, qs, c.dim, c.g, tbl) - stat[tok * q_heads + hq]);
    }
    if (t < s.len)
        mass[((int64_t)seq * c.heads + h) * mass_width + t] += sum;
}

}  // namespace

size_t kv_attention_workspace(int f, const KvCache &c, const KvBatch &b, int q_heads, bool mass)
{
    return mass ? (size_t)b.tokens * q_heads * 4 : 0;
}

hipError_t launch_kv_attention(int f, const KvCache &c, const KvBatch &b, int act_t, const void *q,
                               int64_t qts, int64_t qhs, int q_heads, float scale, int window,
                               void *out, float *lse, float *mass, int64_t mass_width,
                               void *workspace, hipStream_t s)
{
    return kv_by_format(f, [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        kv_attn_simple<F><<<dim3(b.max_new, q_heads, b.seqs), kBlock, 0, s>>>(
            c, b, act_t, (const uint16_t *)q, qts, qhs, q_heads, scale, window, (uint16_t *)out, lse,
            mass ? (float *)workspace : nullptr);
        if (mass)
            kv_mass_simple<F><<<dim3((b.max_len + kBlock - 1) / kBlock, c.heads, b.seqs), kBlock, 0, s>>>(
                c, b, act_t, (const uint16_t *)q, qts, qhs, q_heads, scale, window,
                (const float *)workspace, mass, mass_width);
        return hipGetLastError();
    });
}

}  // namespace q4
