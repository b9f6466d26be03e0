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
// joined by cross-lane maxima.  Keys and values go in one launch: the grid
// counts sequences (z), heads of keys and of values (y) and stretches of new
// tokens (x), so a workgroup's rows lie next to each other in the cache and
// nothing but the page is looked up a lane.  A lane takes four rows where there
// are many, which puts four chains of dependent loads (page, row) in flight.
//
// Bound: reading, HBM traffic: 16 x 4096 tokens of 8 heads of 128, INT4-asym
// g32, 57 us for 354 MB (6.2 TB/s, where a large copy reaches 5.2 and a read
// 6.2).  Appending, vector-ALU issue (the division and the code of every
// value): 8191 NF4 g64 tokens of 32 heads of 128 43 us, 4.0 TB/s, 80 % of the
// slots; 4 prompts of up to 2048 INT4-asym g32 tokens of 8 heads 13.3 us, 2.8
// TB/s, 62 % (short enough that a tenth of it is the launch's ramp).
#include "kv_common.hpp"
#include "q4_code.hpp"

namespace q4 {
namespace {

constexpr int kBlock = 256;
// Rows a lane works on, and from how many pieces of 8 values on (16 x 4096
// INT4-asym tokens of 8 heads read in 1, 2, 4, 8 rows a lane: 84, 68, 58, 56 us;
// 8191 NF4 tokens of 32 heads appended: 61, 50, 43, 43 and read: 39, 31, 28, 36;
// 1024 tokens of 8 heads read in 1 and 4: 3.9 and 4.0.  Calls in 1 and 4, INT4-asym
// tokens of 8 heads of 128: 2^19 pieces alike, 2^20 appended 7.5 and 7.5, read 6.2
// and 5.9; 2^21 12.2 and 11.5, 9.1 and 8.2).
constexpr int kRowsMany = 4;
constexpr int64_t kManyItems = 1 << 20;

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

// What a lane works on: 8 values of a new token's row, U rows at a time so
// that their loads (page, then row) are in flight together.
struct Item {
    int tok, chunk;
    bool in;
    int64_t row;  // in the pool, or -1
};
template <int U>
__device__ __forceinline__ void items_of(Item (&t)[U], const KvCache &c, const KvBatch &b, const KvSeq &s, int seq,
                                         int h, int chunk_shift)
{
    const int32_t *table = b.table + (int64_t)seq * b.table_width;
    int page[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = ((int64_t)blockIdx.x * U + u) * blockDim.x + threadIdx.x;
        t[u].chunk = (int)(i & ((1 << chunk_shift) - 1));
        t[u].tok = (int)(i >> chunk_shift);
        const int pos = s.len - s.fresh + t[u].tok;
        t[u].in = t[u].tok < s.fresh;
        const bool there = t[u].in && pos >= 0;
        page[u] = table[there ? pos >> c.page_shift : 0];
        t[u].row = there ? pos & ((1 << c.page_shift) - 1) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        t[u].row = t[u].row >= 0 && (unsigned)page[u] < (unsigned)c.pages
                       ? (((int64_t)page[u] * c.heads + h) << c.page_shift) + t[u].row
                       : -1;
}

// Codes 8 values, `raw`, of row t and stores them.
template <int FMT, int IN, int LPG>
__device__ __forceinline__ void code_row(const KvCache &c, const KvHalf &to, const Item &t, const u32x4 &raw,
                                         const NF4Bucket *buckets)
{
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
        lo = group_min<LPG>(lo);
        hi = group_max<LPG>(hi);
        // (the constant reciprocal is checked for differences of fp16 values)
        const float q = IN == Q4_F16 ? div_mk(hi - lo, 15.0f, kInv15) : (hi - lo) / 15.0f;
        const uint32_t sb = f2h_bits(keep_f32(fminf(q, 65504.0f)));
        const float d = h2f(sb);
        int z = 0;
        if (d != 0.0f) {
            const float r = rcp_rn(d);
            z = (int)fminf(fmaxf(__builtin_rintf(div_mk(-lo, d, r)), 0.0f), 15.0f);
            const float lo_c = kRint - (float)z;
            uint32_t q8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q8[i] = code_bits(div_mk(x[i], d, r), lo_c, lo_c + 15.0f);
            word = pack8(q8, kRintBias - (uint32_t)z);
        }
        // the odd group's zero-point joins the even one's byte
        const int z1 = __shfl_down(z, LPG);
        if (first && t.row >= 0) {
            ((uint16_t *)to.scales)[t.row * groups + j] = (uint16_t)sb;
            if ((j & 1) == 0)
                to.zeros[t.row * kv_zero_bytes(c.dim, c.g) + (j >> 1)] =
                    (uint8_t)(z | (j + 1 < groups ? z1 << 4 : 0));
        }
    } else {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a = fmaxf(a, fabsf(x[i]));
        a = group_max<LPG>(a);
        if constexpr (FMT == Q4_INT4_SYM) {
            const uint32_t sb = f2h_bits(keep_f32(fminf(div_mk(a, 7.0f, kInv7), 65504.0f)));
            const float d = h2f(sb);
            if (d != 0.0f) {
                const float r = rcp_rn(d);
                uint32_t q8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q8[i] = code_bits(div_mk(x[i], d, r), kRint - 8.0f, kRint + 7.0f);
                word = pack8(q8, kRintBias - 8u);
            } else {
                word = 0x88888888u;
            }
            if (first && t.row >= 0)
                ((uint16_t *)to.scales)[t.row * groups + j] = (uint16_t)sb;
        } else {
            if (first && t.row >= 0)
                ((float *)to.scales)[t.row * groups + j] = a;
            if (IN == Q4_BF16 && !(a >= 0x1p-100f && a <= 0x1p100f) && a != 0.0f) {
                // the reciprocal of so small or large a bf16 absmax is not a
                // normal number: divide both by a power of two (values this
                // takes out of range code as 0 either way)
                const float k2 = a < 1.0f ? 0x1p100f : 0x1p-100f;
                a *= k2;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] *= k2;
            }
            if constexpr (FMT == Q4_NF4)
                word = a != 0.0f ? nf4_word(x, a, buckets) : 0x77777777u;
            else
                word = a != 0.0f ? fp4_word(x, a) : 0u;
        }
    }
    if (t.row >= 0)
        *(uint32_t *)(to.codes + t.row * (c.dim >> 1) + 4 * t.chunk) = word;
}

template <int FMT, int IN, int LPG, int U>
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
    const int seq = blockIdx.z, half = blockIdx.y & 1, h = blockIdx.y >> 1;
    const KvSeq s = kv_seq(b, seq);
    if (s.fresh == 0)
        return;
    const uint16_t *from = half ? v + (int64_t)h * vhs : k + (int64_t)h * khs;
    const int64_t ts = half ? vts : kts;
    // every lane of a row has the same token, so a group works as one; what
    // has no place in the cache reads a row that is there and stores nothing
    Item t[U];
    items_of(t, c, b, s, seq, h, chunk_shift);
    u32x4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        raw[u] = __builtin_nontemporal_load(
            (const u32x4 *)(from + (s.first + min(t[u].tok, s.fresh - 1)) * ts + 8 * t[u].chunk));
#pragma unroll
    for (int u = 0; u < U; ++u)
        code_row<FMT, IN, LPG>(c, half ? c.v : c.k, t[u], raw[u], buckets);
}

template <int FMT, int OUT, int U>
__global__ __launch_bounds__(kBlock) void kv_read_kernel(KvCache c, KvBatch b, uint16_t *__restrict__ k,
                                                         uint16_t *__restrict__ v, int chunk_shift)
{
    __shared__ float2 pairs[f32_absmax(FMT) ? 256 : 1];  // the two levels of a byte
    if constexpr (f32_absmax(FMT)) {
        const float *tbl = FMT == Q4_NF4 ? c_nf4 : c_fp4;
        for (int i = threadIdx.x; i < 256; i += blockDim.x)
            pairs[i] = float2{tbl[i & 15], tbl[i >> 4]};
        __syncthreads();
    }
    const int seq = blockIdx.z, half = blockIdx.y & 1, h = blockIdx.y >> 1;
    const KvSeq s = kv_seq(b, seq);
    Item t[U];
    items_of(t, c, b, s, seq, h, chunk_shift);
    const KvHalf &from = half ? c.v : c.k;
    const int groups = c.dim / c.g;
    uint32_t w[U];
    float sc[U], z[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = max(t[u].row, (int64_t)0);  // (page 0 is read and not used)
        const int j = 8 * t[u].chunk / c.g;
        w[u] = *(const uint32_t *)(from.codes + row * (c.dim >> 1) + 4 * t[u].chunk);
        sc[u] = kv_scale<FMT>(from, row, groups, j);
        z[u] = kv_zero<FMT>(from, row, groups, j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        u32x4 o;
        // one binary32 product each, then one rounding; INT4's is an fma,
        // c s - z s with z s exact: the same single rounding of (c - z) s
        const uint32_t lo = w[u] & 0x0f0f0f0fu, hi = (w[u] >> 4) & 0x0f0f0f0fu;
        const float off = -z[u] * sc[u];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float l0, l1;
            if constexpr (f32_absmax(FMT)) {
                const float2 p = pairs[(w[u] >> (8 * i)) & 255];
                l0 = keep_f32(p.x * sc[u]);
                l1 = keep_f32(p.y * sc[u]);
            } else {
                l0 = __builtin_fmaf((float)((lo >> (8 * i)) & 255u), sc[u], off);
                l1 = __builtin_fmaf((float)((hi >> (8 * i)) & 255u), sc[u], off);
            }
            o[i] = OUT == Q4_F16 ? pack_h2(l0, l1) : pack_bf2(l0, l1);
        }
        if (t[u].row < 0)
            o = u32x4{0, 0, 0, 0};
        if (t[u].in)
            __builtin_nontemporal_store(o, (u32x4 *)((half ? v : k) +
                                                     ((int64_t)(s.first + t[u].tok) * c.heads + h) * c.dim +
                                                     8 * t[u].chunk));
    }
}

struct Launch {
    dim3 grid;
    int block, shift;
    bool many;  // kRowsMany rows a lane
};
Launch launch_of(const KvCache &c, const KvBatch &b)
{
    Launch l;
    l.shift = __builtin_ctz(c.dim / 8);
    const int64_t items = (int64_t)b.max_new << l.shift;
    // (single tokens leave most of a large workgroup idle: 64 sequences of 8
    // heads appended in 2.4 us, in workgroups of 256 2.6)
    l.block = items <= 64 ? 64 : kBlock;
    l.many = items * 2 * c.heads * b.seqs >= kManyItems;
    const int64_t per = (int64_t)l.block * (l.many ? kRowsMany : 1);
    l.grid = dim3((unsigned)((items + per - 1) / per), (unsigned)(2 * c.heads), (unsigned)b.seqs);
    return l;
}

}  // namespace

hipError_t launch_kv_append(int f, const KvCache &c, const KvBatch &b, int in_t, const void *k,
                            int64_t kts, int64_t khs, const void *v, int64_t vts, int64_t vhs,
                            hipStream_t s)
{
    return kv_by_format(f, [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        const Launch l = launch_of(c, b);
        auto launch = [&](auto in, auto lpg, auto rows) {
            kv_append_kernel<F, decltype(in)::value, decltype(lpg)::value, decltype(rows)::value>
                <<<l.grid, l.block, 0, s>>>(c, b, (const uint16_t *)k, kts, khs, (const uint16_t *)v, vts, vhs,
                                            l.shift);
            return hipGetLastError();
        };
        auto go = [&](auto in, auto lpg) {
            return l.many ? launch(in, lpg, KvInt<kRowsMany>{}) : launch(in, lpg, KvInt<1>{});
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
        const Launch l = launch_of(c, b);
        auto launch = [&](auto out, auto rows) {
            kv_read_kernel<F, decltype(out)::value, decltype(rows)::value>
                <<<l.grid, l.block, 0, s>>>(c, b, (uint16_t *)k, (uint16_t *)v, l.shift);
            return hipGetLastError();
        };
        auto go = [&](auto out) { return l.many ? launch(out, KvInt<kRowsMany>{}) : launch(out, KvInt<1>{}); };
        return out_t == Q4_F16 ? go(KvInt<Q4_F16>{}) : go(KvInt<Q4_BF16>{});
    });
}

}  // namespace q4
