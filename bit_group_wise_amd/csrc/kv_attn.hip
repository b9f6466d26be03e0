// kv_attn.hip -- q4_kv_attention: which kernel takes a call, the workspace, and
// the sum of a split range's parts.
#include "kv_attn.hpp"

namespace q4 {
namespace {

// Joins the parts of a row: one workgroup per new token and query head.
template <int D>
__global__ __launch_bounds__(D) void kv_join_kernel(KvBatch b, Rows rows, Split sp, const float *__restrict__ part,
                                                    const float2 *__restrict__ part_ml)
{
    const int seq = blockIdx.z, head = blockIdx.y, tok = blockIdx.x, d = threadIdx.x;
    const KvSeq s = kv_seq(b, seq);
    if (tok >= s.fresh)
        return;
    const int64_t to = (int64_t)(s.first + tok) * rows.q_heads + head;
    // the parts up to the one that holds the row's own position
    const int seen = s.len - s.fresh + tok + 1 - range_begin(s, rows.window);
    const int n = max(1, (seen + sp.span - 1) / sp.span);
    const float2 *ml = part_ml + to * sp.parts;
    float m = kNone;
    for (int p = 0; p < n; ++p)
        m = fmaxf(m, ml[p].x);
    float sum = 0.0f, l = 0.0f;
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
        const float f = __builtin_amdgcn_exp2f(ml[p].x - m);
        l += ml[p].y * f;
        sum += part[(to * sp.parts + p) * D + d] * f;
    }
    const float v = l > 0.0f ? sum / l : 0.0f;
    rows.out[to * D + d] = (uint16_t)(rows.act == Q4_F16 ? f2h_bits(v) : f2bf_bits(v));
    if (d == 0) {
        const float e = l > 0.0f ? m + __builtin_amdgcn_logf(l) : -__builtin_inff();
        if (rows.lse)
            rows.lse[to] = e * kLn2;
        if (rows.stat)
            rows.stat[to] = e;
    }
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// A head's rows by scale groups fill the columns of the token kernel's tiles;
// what does not fit goes to the prompt kernel.
bool is_prompt(const KvCache &c, const KvBatch &b, int group) { return (int64_t)b.max_new * group > few_rows(c); }

Split split_for(const KvCache &c, const KvBatch &b, int group, int window)
{
    return is_prompt(c, b, group) ? prompt_split(c, b, group, window) : token_split(c, b, group, window);
}

}  // namespace

size_t kv_attention_workspace(const KvCache &c, const KvBatch &b, int q_heads, int window, bool mass)
{
    const Split sp = split_for(c, b, q_heads / c.heads, window);
    const size_t rows = (size_t)b.tokens * q_heads;
    size_t n = 0;
    if (sp.parts > 1)
        n = round256(rows * sp.parts * sizeof(float2)) + rows * sp.parts * c.dim * 4;
    // (the parts are done with when the mass pass starts)
    return mass ? round256(rows * 4) + std::max(n, kv_mass_workspace(c, b, q_heads / c.heads)) : n;
}

hipError_t launch_kv_attention(int f, const KvCache &c, const KvBatch &b, int act_t, const void *q,
                               int64_t qts, int64_t qhs, int q_heads, float scale, int window,
                               void *out, float *lse, float *mass, int64_t mass_width,
                               void *workspace, hipStream_t s)
{
    const int group = q_heads / c.heads;
    const Split sp = split_for(c, b, group, window);
    const size_t n = (size_t)b.tokens * q_heads;
    char *w = (char *)workspace;
    Rows rows{(const uint16_t *)q, qts, qhs, q_heads, group, act_t, window, scale * kLog2e,
              (uint16_t *)out, lse, nullptr};
    if (mass) {
        rows.stat = (float *)w;
        w += round256(n * 4);
    }
    float2 *part_ml = (float2 *)w;
    float *part = (float *)(w + round256(n * sp.parts * sizeof(float2)));
    hipError_t e = is_prompt(c, b, group) ? launch_kv_prompt(f, c, b, rows, sp, part, part_ml, s)
                                       : launch_kv_token(f, c, b, rows, sp, part, part_ml, s);
    if (e != hipSuccess)
        return e;
    if (sp.parts > 1) {
        const dim3 grid(b.max_new, q_heads, b.seqs);
        if (c.dim == 64)
            kv_join_kernel<64><<<grid, 64, 0, s>>>(b, rows, sp, part, part_ml);
        else if (c.dim == 128)
            kv_join_kernel<128><<<grid, 128, 0, s>>>(b, rows, sp, part, part_ml);
        else
            kv_join_kernel<256><<<grid, 256, 0, s>>>(b, rows, sp, part, part_ml);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return mass ? launch_kv_mass(f, c, b, rows, mass, mass_width, w, s) : hipSuccess;
}

}  // namespace q4
