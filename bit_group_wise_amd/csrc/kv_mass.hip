// kv_mass.hip -- the attention weight that each cached token draws, added to
// its mass (q4_kv_attention with mass).
//
// A token's mass is a sum over rows of exp(x_t - lse): it needs every row's
// final statistics, so it is a second pass over the keys.  A lane's scores
// belong to one row and several tokens; sums run over rows in the lane and
// then over the 16 columns of a tile, in a fixed order.
#include "kv_attn.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 4;
constexpr int kBlock = 64 * kWaves;
constexpr int kStep = 32;  // tokens per wave

// mass[b, h, t] += sum over rows of 2^(x - stat), one wave per 32 tokens, the
// rows 16 at a time.  A row that sees nothing has stat = -inf and is skipped.
template <int FMT, int D, int GS>
__global__ __launch_bounds__(kBlock) void kv_mass_kernel(KvCache c, KvBatch b, Rows rows,
                                                         float *__restrict__ mass, int64_t mass_width)
{
    __shared__ uint32_t pairs[FMT == Q4_NF4 ? 256 : 1];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int seq = blockIdx.z, h = blockIdx.y;
    const KvSeq s = kv_seq(b, seq);
    if constexpr (FMT == Q4_NF4) {
        pairs[tid] = nf4_pair(tid);
        __syncthreads();
    }
    const int t0 = range_begin(s, rows.window) + ((int)blockIdx.x * kWaves + wave) * kStep;
    if (t0 >= s.len)
        return;
    Pages pg{b.table + (int64_t)seq * b.table_width, c.page_shift, c.heads, h, c.pages, -1000,
             (s.len - 1) >> c.page_shift, -1};
    Tile<FMT, D, GS> t[2];
    t[0].load(c, pg.row(t0, s.len, lane), lane);
    t[1].load(c, pg.row(t0 + 16, s.len, lane), lane);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int nrows = s.fresh * rows.group;
    for (int r0 = 0; r0 < nrows; r0 += 16) {
        const int row = r0 + i;
        const bool live = row < nrows;
        const int tok = live ? row / rows.group : 0;
        const int head = h * rows.group + (live ? row - tok * rows.group : 0);
        const int pos = live ? s.len - s.fresh + tok : -1;
        const int low = rows.window > 0 ? pos - rows.window : -1;
        Queries<FMT, D, GS> q;
        q.load(rows.q + (int64_t)(s.first + tok) * rows.qts + (int64_t)head * rows.qhs, live, rows.act,
               rows.scale2, kg);
        const float st = live ? rows.stat[(int64_t)(s.first + tok) * rows.q_heads + head] : 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const f32x4 a = scores<FMT, D, GS>(t[u], q, pairs);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int at = t0 + 16 * u + 4 * kg + r;
                const bool see = t[u].there && at <= pos && at > low;
                sum[4 * u + r] += see ? __builtin_amdgcn_exp2f(__builtin_fmaf(a[r], q.factor, -st)) : 0.0f;
            }
        }
    }
    // over the 16 columns, in a fixed order
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int d = 1; d < 16; d <<= 1)
            sum[e] += __shfl_xor(sum[e], d);
    if (i < 8) {
        float v = sum[0];
#pragma unroll
        for (int e = 1; e < 8; ++e)
            v = i == e ? sum[e] : v;
        const int at = t0 + 16 * (i >> 2) + 4 * kg + (i & 3);
        if (at < s.len)
            mass[((int64_t)seq * c.heads + h) * mass_width + at] += v;
    }
}

}  // namespace

hipError_t launch_kv_mass(int f, const KvCache &c, const KvBatch &b, const Rows &rows, float *mass,
                          int64_t mass_width, hipStream_t s)
{
    const int64_t range = longest_range(b, rows.window);
    const int per = kWaves * kStep;
    return kv_by_shape(f, c.dim, c.g, [&](auto fmt, auto dim, auto gs) {
        kv_mass_kernel<decltype(fmt)::value, decltype(dim)::value, decltype(gs)::value>
            <<<dim3((unsigned)((range + per - 1) / per), c.heads, b.seqs), kBlock, 0, s>>>(c, b, rows, mass,
                                                                                           mass_width);
        return hipGetLastError();
    });
}

}  // namespace q4
