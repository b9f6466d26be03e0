// kv_attn.hip -- q4_kv_attention: which kernel takes a call, the workspace, and
// the sum of a split range's parts (4 to 6 us for the split calls that
// kv_token.hip lists, 9 us for 32768 rows in two parts: a launch and
// the latency of two dependent reads).
#include "kv_attn.hpp"

namespace q4 {
namespace {

constexpr int kJoin = 256;

// Joins the parts of a row (a new token's query head): D / 4 lanes a part,
// TEAMS parts at a time.  Many parts are shared by a workgroup's teams; few
// are summed by one team, the workgroup taking several rows (whole calls: 96
// parts of one token's 32 rows 33 us by teams, 47 by one team; 3 parts of 32
// tokens 31.4 by one team, 31.0 by teams; 2 parts of 2048 rows 109 by one team,
// 119 by teams).
template <int D, bool MANY>
__global__ __launch_bounds__(kJoin) void kv_join_kernel(KvBatch b, Rows rows, Split sp, const float *__restrict__ part,
                                                        const float2 *__restrict__ part_ml)
{
    constexpr int LANES = D / 4, TEAMS = MANY ? kJoin / LANES : 1, RPB = kJoin / (LANES * TEAMS);
    __shared__ f32x4 sums[MANY ? TEAMS : 1][LANES];
    __shared__ float ls[TEAMS];
    const int seq = blockIdx.z, head = blockIdx.y, tok = blockIdx.x * RPB + threadIdx.x / (LANES * TEAMS);
    const int team = threadIdx.x / LANES % TEAMS, d = threadIdx.x % LANES;
    const KvSeq s = kv_seq(b, seq);
    if (tok >= s.fresh)
        return;
    const int64_t to = (int64_t)(s.first + tok) * rows.q_heads + head;
    // the parts up to the one that holds the row's own position
    const int seen = s.len - s.fresh + tok + 1 - range_begin(s, rows.window);
    const int n = max(1, (seen + sp.span - 1) / sp.span);
    const float2 *ml = part_ml + to * sp.parts;
    float m = kNone;
    if constexpr (MANY) {
        for (int p = threadIdx.x & 63; p < n; p += 64)
            m = fmaxf(m, ml[p].x);
#pragma unroll
        for (int e = 1; e < 64; e <<= 1)
            m = fmaxf(m, __shfl_xor(m, e));
    } else {
        for (int p = 0; p < n; ++p)
            m = fmaxf(m, ml[p].x);
    }
    f32x4 sum = {0, 0, 0, 0};
    float l = 0.0f;
#pragma unroll 4
    for (int p = team; p < n; p += TEAMS) {
        const float2 e = ml[p];
        const float f = __builtin_amdgcn_exp2f(e.x - m);
        l += e.y * f;
        sum += *(const f32x4 *)(part + (to * sp.parts + p) * D + 4 * d) * f;
    }
    if constexpr (MANY) {
        sums[team][d] = sum;
        if (d == 0)
            ls[team] = l;
        __syncthreads();
        if (team)
            return;
#pragma unroll
        for (int e = 1; e < TEAMS; ++e) {
            sum += sums[e][d];
            l += ls[e];
        }
    }
    sum *= l > 0.0f ? 1.0f / l : 0.0f;
    u32x2 pk;
    pk[0] = rows.act == Q4_F16 ? pair_h2(sum[0], sum[1]) : pack_bf2(sum[0], sum[1]);
    pk[1] = rows.act == Q4_F16 ? pair_h2(sum[2], sum[3]) : pack_bf2(sum[2], sum[3]);
    *(u32x2 *)(rows.out + to * D + 4 * d) = pk;
    if (d == 0) {
        const float e = l > 0.0f ? row_stat(m, l) : -__builtin_inff();
        if (rows.lse)
            rows.lse[to] = e * kLn2;
        if (rows.stat)
            rows.stat[to] = e;
    }
}

template <int D>
void join(const KvBatch &b, const Rows &rows, const Split &sp, const float *part, const float2 *part_ml, hipStream_t s)
{
    constexpr int RPB = kJoin / (D / 4);
    if (sp.parts > 4)
        kv_join_kernel<D, true><<<dim3(b.max_new, rows.q_heads, b.seqs), kJoin, 0, s>>>(b, rows, sp, part, part_ml);
    else
        kv_join_kernel<D, false><<<dim3((b.max_new + RPB - 1) / RPB, rows.q_heads, b.seqs), kJoin, 0, s>>>(b, rows, sp, part,
                                                                                                     part_ml);
}

// A window that no sequence outgrows is none: positions less a window then stay
// far inside 32 bits, also where a sequence has more new tokens than cached ones.
int window_of(const KvBatch &b, int window) { return window < b.max_len ? window : 0; }

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
    window = window_of(b, window);
    const Split sp = split_for(c, b, q_heads / c.heads, window);
    const size_t rows = (size_t)b.tokens * q_heads;
    size_t n = 0;
    if (sp.parts > 1)
        n = round256(rows * sp.parts * sizeof(float2)) + rows * sp.parts * c.dim * 4;
    // (the parts are done with when the mass pass starts)
    const int group = q_heads / c.heads;
    return mass ? round256(rows * 4) + round256(kv_kept_bytes(c, b, group, window)) +
                      std::max(n, kv_mass_workspace(c, b, group))
                : n;
}

hipError_t launch_kv_attention(int f, const KvCache &c, const KvBatch &b, int act_t, const void *q,
                               int64_t qts, int64_t qhs, int q_heads, float scale, int window,
                               void *out, float *lse, float *mass, int64_t mass_width,
                               void *workspace, hipStream_t s)
{
    const int group = q_heads / c.heads;
    window = window_of(b, window);
    const Split sp = split_for(c, b, group, window);
    const size_t n = (size_t)b.tokens * q_heads;
    char *w = (char *)workspace;
    Rows rows{(const uint16_t *)q, qts, qhs, q_heads, group, act_t, window, scale * kLog2e,
              (uint16_t *)out, lse, nullptr, nullptr, 0, 0};
    if (mass) {
        rows.stat = (float *)w;
        w += round256(n * 4);
        if (const size_t kept = kv_kept_bytes(c, b, group, window)) {
            rows.kept = (float *)w;
            rows.kept_range = longest_range(b, window);
            rows.kept_rows = b.max_new * group;
            w += round256(kept);
        }
    }
    float2 *part_ml = (float2 *)w;
    float *part = (float *)(w + round256(n * sp.parts * sizeof(float2)));
    const auto launch = is_prompt(c, b, group) ? launch_kv_prompt : act_t == Q4_F16 ? launch_kv_token_f16 : launch_kv_token;
    hipError_t e = launch(f, c, b, rows, sp, part, part_ml, s);
    if (e != hipSuccess)
        return e;
    if (sp.parts > 1) {
        if (c.dim == 64)
            join<64>(b, rows, sp, part, part_ml, s);
        else if (c.dim == 128)
            join<128>(b, rows, sp, part, part_ml, s);
        else
            join<256>(b, rows, sp, part, part_ml, s);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return mass ? launch_kv_mass(f, c, b, rows, mass, mass_width, w, s) : hipSuccess;
}

}  // namespace q4
