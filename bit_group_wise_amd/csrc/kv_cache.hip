// kv_cache.hip -- new tokens into the 4-bit key/value cache, and rows back out
// of it as 16-bit values (q4_kv_append, q4_kv_read).
//
// Method: the coding rules of q4_quantize on rows of `dim` values ("Block-wise
// quantisation, stated exactly"; "How 4-bit quantization works"; "INT4", "How
// it works" / "Components"): per group of g values the absmax or the
// zero-anchored range, the stored scale, one IEEE binary32 division a value,
// the nearest level; and q4_dequantize's product back.
//
// gfx950 mapping: a lane owns 8 consecutive values (16 bytes in, one dword of
// codes out), so a row is dim / 8 lanes and a group g / 8 adjacent lanes
// joined by cross-lane maxima.  Keys and values of a sequence go in one
// launch: the grid's y counts sequences, x their (key | value, token, head,
// chunk) in order, so that neighbouring lanes read neighbouring bytes.
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
// NF4's decision thresholds (see q4_common.hpp): the code of x is the number
// of thresholds at or below it.
__constant__ NF4Bucket c_buckets[33] = {
#define B(i) {kNF4Buckets.e[i].thr, kNF4Buckets.e[i].base}
    B(0),  B(1),  B(2),  B(3),  B(4),  B(5),  B(6),  B(7),  B(8),  B(9),  B(10),
    B(11), B(12), B(13), B(14), B(15), B(16), B(17), B(18), B(19), B(20), B(21),
    B(22), B(23), B(24), B(25), B(26), B(27), B(28), B(29), B(30), B(31), B(32),
#undef B
};

template <int LPG>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int d = 1; d < LPG; d <<= 1)
        v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// (key | value, token, head, chunk of 8 values) of item i of a sequence.
struct Item {
    int half, tok, head, chunk;
    bool in;
};
__device__ __forceinline__ Item item_of(int64_t i, int fresh, int heads, int chunk_shift)
{
    Item t;
    t.chunk = (int)(i & ((1 << chunk_shift) - 1));
    const int64_t row = i >> chunk_shift;
    const int64_t tok = row / heads;
    t.head = (int)(row - tok * heads);
    t.in = tok < 2 * (int64_t)fresh;
    t.half = tok >= fresh;
    t.tok = (int)(t.half ? tok - fresh : tok);
    return t;
}

template <int FMT, int IN, int LPG>
__global__ __launch_bounds__(kBlock) void kv_append_kernel(
    KvCache c, KvBatch b, const uint16_t *__restrict__ k, int64_t kts, int64_t khs,
    const uint16_t *__restrict__ v, int64_t vts, int64_t vhs, int chunk_shift)
{
    __shared__ NF4Bucket buckets[FMT == Q4_NF4 ? 33 : 1];
    if constexpr (FMT == Q4_NF4) {
        if (threadIdx.x < 33)
            buckets[threadIdx.x] = c_buckets[threadIdx.x];
        __syncthreads();
    }
    const int seq = blockIdx.y;
    const KvSeq s = kv_seq(b, seq);
    const Item t = item_of((int64_t)blockIdx.x * kBlock + threadIdx.x, s.fresh, c.heads, chunk_shift);
    const int pos = s.len - s.fresh + t.tok;
    // every lane of a group has the same token, so a group leaves as one
    if (!t.in || pos < 0)
        return;
    const int64_t row = kv_row(c, b.table + (int64_t)seq * b.table_width, pos, t.head);
    if (row < 0)
        return;
    const KvHalf &to = t.half ? c.v : c.k;
    const int64_t src = (int64_t)(s.first + t.tok) * (t.half ? vts : kts) +
                        (int64_t)t.head * (t.half ? vhs : khs) + 8 * t.chunk;
    const u32x4 raw = *(const u32x4 *)((t.half ? v : k) + src);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (IN == Q4_F16) {
            x[2 * i] = h2f(raw[i] & 0xffffu);
            x[2 * i + 1] = h2f(raw[i] >> 16);
        } else {
            x[2 * i] = bf2f(raw[i] & 0xffffu);
            x[2 * i + 1] = std::bit_cast<float>(raw[i] & 0xffff0000u);
        }
    }
    const int groups = c.dim / c.g, j = t.chunk / LPG;
    const bool first = t.chunk % LPG == 0;
    uint32_t word = 0;
    if constexpr (FMT == Q4_INT4_ASYM) {
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, x[i]);
            hi = fmaxf(hi, x[i]);
        }
        hi = group_max<LPG>(hi);
        lo = -group_max<LPG>(-lo);
        const uint32_t sb = f2h_bits(fminf((hi - lo) / 15.0f, 65504.0f));
        const float d = h2f(sb);
        const float z = d > 0.0f ? fminf(fmaxf(rintf(-lo / d), 0.0f), 15.0f) : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = d > 0.0f ? fminf(fmaxf(rintf(x[i] / d) + z, 0.0f), 15.0f) : 0.0f;
            word |= (uint32_t)q << (4 * i);
        }
        // the odd group's zero-point joins the even one's byte
        const float z1 = __shfl_down(z, LPG);
        if (first) {
            ((uint16_t *)to.scales)[row * groups + j] = (uint16_t)sb;
            if ((j & 1) == 0)
                to.zeros[row * kv_zero_bytes(c.dim, c.g) + (j >> 1)] =
                    (uint8_t)((uint32_t)z | (j + 1 < groups ? (uint32_t)z1 << 4 : 0u));
        }
    } else {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a = fmaxf(a, fabsf(x[i]));
        a = group_max<LPG>(a);
        if constexpr (FMT == Q4_INT4_SYM) {
            const uint32_t sb = f2h_bits(fminf(a / 7.0f, 65504.0f));
            const float d = h2f(sb);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = d > 0.0f ? fminf(fmaxf(rintf(x[i] / d), -8.0f), 7.0f) : 0.0f;
                word |= (uint32_t)(int)(q + 8.0f) << (4 * i);
            }
            if (first)
                ((uint16_t *)to.scales)[row * groups + j] = (uint16_t)sb;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = a > 0.0f ? x[i] / a : 0.0f;
                uint32_t code;
                if constexpr (FMT == Q4_NF4) {
                    const NF4Bucket e = buckets[(int)((q + 1.0f) * 16.0f)];
                    code = e.base + (q >= e.thr ? 1u : 0u);
                } else {
                    code = 0;
#pragma unroll
                    for (int m = 0; m < 7; ++m)
                        code += fabsf(q) >= kFP4Thr[m] ? 1u : 0u;
                    code |= q < 0.0f && code ? 8u : 0u;
                }
                word |= code << (4 * i);
            }
            if (first)
                ((float *)to.scales)[row * groups + j] = a;
        }
    }
    *(uint32_t *)(to.codes + row * (c.dim >> 1) + 4 * t.chunk) = word;
}

template <int FMT, int OUT>
__global__ __launch_bounds__(kBlock) void kv_read_kernel(KvCache c, KvBatch b, uint16_t *__restrict__ k,
                                                         uint16_t *__restrict__ v, int chunk_shift)
{
    __shared__ float tbl[16];
    if constexpr (f32_absmax(FMT)) {
        if (threadIdx.x < 16)
            tbl[threadIdx.x] = FMT == Q4_NF4 ? c_nf4[threadIdx.x] : c_fp4[threadIdx.x];
        __syncthreads();
    }
    const int seq = blockIdx.y;
    const KvSeq s = kv_seq(b, seq);
    const Item t = item_of((int64_t)blockIdx.x * kBlock + threadIdx.x, s.fresh, c.heads, chunk_shift);
    if (!t.in)
        return;
    const int pos = s.len - s.fresh + t.tok;
    const int64_t row =
        pos < 0 ? -1 : kv_row(c, b.table + (int64_t)seq * b.table_width, pos, t.head);
    u32x4 o = {0, 0, 0, 0};
    if (row >= 0) {
        const KvHalf &from = t.half ? c.v : c.k;
        const uint32_t w = *(const uint32_t *)(from.codes + row * (c.dim >> 1) + 4 * t.chunk);
        const int groups = c.dim / c.g, j = 8 * t.chunk / c.g;
        const float sc = kv_scale<FMT>(from, row, groups, j);
        const float z = kv_zero<FMT>(from, row, groups, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // one binary32 product each, then one rounding
            const float p0 = keep_f32((kv_level<FMT>(w >> (8 * i), tbl) - z) * sc);
            const float p1 = keep_f32((kv_level<FMT>(w >> (8 * i + 4), tbl) - z) * sc);
            o[i] = OUT == Q4_F16 ? pack_h2(p0, p1) : pack_bf2(p0, p1);
        }
    }
    *(u32x4 *)((t.half ? v : k) + ((int64_t)(s.first + t.tok) * c.heads + t.head) * c.dim +
               8 * t.chunk) = o;
}

dim3 item_grid(const KvCache &c, const KvBatch &b)
{
    const int64_t items = 2 * (int64_t)b.max_new * c.heads * (c.dim / 8);
    return dim3((unsigned)((items + kBlock - 1) / kBlock), (unsigned)b.seqs);
}

}  // namespace

hipError_t launch_kv_append(int f, const KvCache &c, const KvBatch &b, int in_t, const void *k,
                            int64_t kts, int64_t khs, const void *v, int64_t vts, int64_t vhs,
                            hipStream_t s)
{
    return kv_by_format(f, [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        const int shift = __builtin_ctz(c.dim / 8);
        auto go = [&](auto in, auto lpg) {
            kv_append_kernel<F, decltype(in)::value, decltype(lpg)::value>
                <<<item_grid(c, b), kBlock, 0, s>>>(c, b, (const uint16_t *)k, kts, khs,
                                                    (const uint16_t *)v, vts, vhs, shift);
            return hipGetLastError();
        };
        auto by_g = [&](auto in) {
            return c.g == 32 ? go(in, KvInt<4>{}) : c.g == 64 ? go(in, KvInt<8>{}) : go(in, KvInt<16>{});
        };
        return in_t == Q4_F16 ? by_g(KvInt<Q4_F16>{}) : by_g(KvInt<Q4_BF16>{});
    });
}

hipError_t launch_kv_read(int f, const KvCache &c, const KvBatch &b, int out_t, void *k, void *v,
                          hipStream_t s)
{
    return kv_by_format(f, [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        const int shift = __builtin_ctz(c.dim / 8);
        if (out_t == Q4_F16)
            kv_read_kernel<F, Q4_F16><<<item_grid(c, b), kBlock, 0, s>>>(c, b, (uint16_t *)k, (uint16_t *)v, shift);
        else
            kv_read_kernel<F, Q4_BF16><<<item_grid(c, b), kBlock, 0, s>>>(c, b, (uint16_t *)k, (uint16_t *)v, shift);
        return hipGetLastError();
    });
}

}  // namespace q4
