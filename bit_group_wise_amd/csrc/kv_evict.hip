// kv_evict.hip -- eviction from the 4-bit key/value cache by accumulated
// attention weight (q4_kv_evict).
//
// Select: per (sequence, head) the budget - recent largest masses among the
// tokens before the recent ones.  The masses map to integers of the same
// order; the smallest one kept, T, is found digit by digit (8 bits a pass,
// most significant first) by counting the keys that share the digits found so
// far; the counts are integers, so their atomics' order does not matter.
// Everything above T stays, and of the tokens equal to T the first ones, as
// many as are missing.  A pass over the tokens in order with a running count
// then lists the kept positions.
//
// Move: one lane per 16 bytes of codes copies the kept rows to their new
// pages; rows never move within their old pages, so no order is needed.
#include "kv_common.hpp"

namespace q4 {
namespace {

constexpr int kSel = 1024;
constexpr int kMove = 256;

// Masses as integers of the same order; NaN below everything.
__device__ __forceinline__ uint32_t mass_key(float f)
{
    if (f != f)
        return 0;
    const uint32_t u = std::bit_cast<uint32_t>(f == 0.0f ? 0.0f : f);  // -0 is 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive sum over the workgroup's threads; every thread gets the total.
__device__ __forceinline__ int block_scan(int v, int *wsum, int *total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        v += lane >= d ? o : 0;
    }
    __syncthreads();
    if (lane == 63)
        wsum[wave] = v;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < kSel / 64; ++i) {
        before += i < wave ? wsum[i] : 0;
        all += wsum[i];
    }
    *total = all;
    return v + before;
}

__global__ __launch_bounds__(kSel) void kv_select_kernel(KvCache c, KvBatch b,
                                                         const float *__restrict__ mass, int64_t width,
                                                         int budget, int recent, int32_t *__restrict__ new_lens,
                                                         float *__restrict__ new_mass, int64_t new_width,
                                                         int32_t *__restrict__ kept)
{
    __shared__ int hist[256], wsum[kSel / 64];
    __shared__ uint32_t sh_key;
    __shared__ int sh_need;
    const int h = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x;
    const int len = min(max(b.lens[seq], 0), b.max_len);
    const int64_t rowid = (int64_t)seq * c.heads + h;
    const float *m = mass + rowid * width;
    float *mo = new_mass + rowid * new_width;
    int32_t *ko = kept + rowid * budget;
    const int n = min(len, budget);
    if (h == 0 && tid == 0)
        new_lens[seq] = n;
    if (len <= budget) {
        for (int64_t i = tid; i < new_width; i += kSel)
            mo[i] = i < n ? m[i] : 0.0f;
        for (int i = tid; i < budget; i += kSel)
            ko[i] = i < n ? i : -1;
        return;
    }
    const int old = len - recent, want = budget - recent;  // want < old
    uint32_t T = 0;
    int need = want;  // tokens equal to T (in the digits found) still to take
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSel)
            hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int t = tid; t < old; t += kSel) {
            const uint32_t k = mass_key(m[t]);
            if ((k & mask) == T)
                atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, d = 255;
            while (d > 0 && hist[d] < left)
                left -= hist[d--];
            sh_key = T | (uint32_t)d << shift;
            sh_need = left;
        }
        __syncthreads();
        T = sh_key;
        need = sh_need;
        __syncthreads();
    }
    int done = 0, ties = 0;  // kept, and tokens equal to T seen, before this stretch
    for (int t0 = 0; t0 < len; t0 += kSel) {
        const int t = t0 + tid;
        const float f = t < len ? m[t] : 0.0f;
        const uint32_t k = mass_key(f);
        const bool tie = t < old && k == T;
        int total;
        const int rank = block_scan(tie, wsum, &total);
        const bool stay = t < len && (t >= old || k > T || (tie && ties + rank <= need));
        ties += total;
        const int place = done + block_scan(stay, wsum, &total) - 1;
        if (stay) {
            ko[place] = t;
            mo[place] = f;
        }
        done += total;
    }
    for (int64_t i = n + tid; i < new_width; i += kSel)
        mo[i] = 0.0f;
}

__global__ __launch_bounds__(kMove) void kv_move_kernel(KvCache c, KvBatch b,
                                                        const int32_t *__restrict__ new_table, int new_tw,
                                                        int budget, const int32_t *__restrict__ kept,
                                                        int row_scale_bytes, int row_zero_bytes, int chunk_shift)
{
    const int h = blockIdx.y, seq = blockIdx.z;
    const int64_t item = (int64_t)blockIdx.x * kMove + threadIdx.x;
    const int chunk = (int)(item & ((1 << chunk_shift) - 1));
    const int64_t place = item >> chunk_shift;
    if (place >= budget)
        return;
    const int t = kept[((int64_t)seq * c.heads + h) * budget + place];
    if (t < 0)
        return;
    const int64_t src = kv_row(c, b.table + (int64_t)seq * b.table_width, t, h);
    const int64_t dst = kv_row(c, new_table + (int64_t)seq * new_tw, (int)place, h);
    if (src < 0 || dst < 0)
        return;
    const int row_bytes = c.dim >> 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const KvHalf &x = i ? c.v : c.k;
        *(u32x4 *)(x.codes + dst * row_bytes + 16 * chunk) =
            *(const u32x4 *)(x.codes + src * row_bytes + 16 * chunk);
        if (chunk == 0) {
            const uint16_t *s = (const uint16_t *)((const char *)x.scales + src * row_scale_bytes);
            uint16_t *d = (uint16_t *)((char *)x.scales + dst * row_scale_bytes);
            for (int j = 0; j < row_scale_bytes / 2; ++j)
                d[j] = s[j];
            for (int j = 0; j < row_zero_bytes; ++j)
                x.zeros[dst * row_zero_bytes + j] = x.zeros[src * row_zero_bytes + j];
        }
    }
}

}  // namespace

hipError_t launch_kv_evict(int f, const KvCache &c, const KvBatch &b, const float *mass,
                           int64_t mass_width, const int32_t *new_table, int new_table_width,
                           int budget, int recent, int32_t *new_lens, float *new_mass,
                           int64_t new_width, int32_t *kept, hipStream_t s)
{
    kv_select_kernel<<<dim3(c.heads, b.seqs), kSel, 0, s>>>(c, b, mass, mass_width, budget, recent,
                                                           new_lens, new_mass, new_width, kept);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int shift = __builtin_ctz(c.dim / 32);
    const int64_t items = (int64_t)budget << shift;
    const int groups = c.dim / c.g;
    kv_move_kernel<<<dim3((unsigned)((items + kMove - 1) / kMove), c.heads, b.seqs), kMove, 0, s>>>(
        c, b, new_table, new_table_width, budget, kept, groups * (f32_absmax(f) ? 4 : 2),
        f == Q4_INT4_ASYM ? kv_zero_bytes(c.dim, c.g) : 0, shift);
    return hipGetLastError();
}

}  // namespace q4
