// kv_evict.hip -- eviction from the 4-bit key/value cache by accumulated
// attention weight (q4_kv_evict).
//
// Select: per (sequence, head) the budget - recent largest masses among the
// tokens before the recent ones.  The masses map to integers of the same
// order; the smallest one kept, T, is the largest integer that at least that
// many keys reach, found two bits at a time by counting the keys at or above
// three candidates.  Everything above T stays, and of the tokens equal to T
// the first ones, as many as are missing.  A workgroup's threads hold runs of
// consecutive tokens, so two running counts over the threads give every kept
// token's place.  Counting needs no atomics: a wave counts by ballot, and the
// waves' counts meet in LDS.  Tokens whose page does not exist are not there:
// they are no candidates, and the recent ones are the last that are.
//
// Bound: latency.  A pass over the candidates is some 500 cycles of ballots, a
// barrier and the exchange in LDS, whatever the length: 12 us for 1088 tokens
// in four waves, 24 us for 16 x 8 rows of 8192 in sixteen.
//
// Move: rows go to other pages, so no order is needed: a lane copies 16 bytes
// of a row's codes, and a row's lanes share its scales and zero-points.  Bound:
// HBM traffic.  Kept tokens lie among dropped ones and a row of codes is half a
// 128-byte line (dim 128), so more is read than written: 16 x 4096 of 8192
// tokens, 8 heads of 128, INT4-asym g32 36.8 us, 113 MB read and 78 MB written
// (counted), 5.2 TB/s, what a large copy reaches.
#include <algorithm>

#include "kv_common.hpp"

namespace q4 {
namespace {

constexpr int kSel = 1024;
constexpr int kSelFew = 256;
constexpr int kMove = 256;
// Rows a lane moves, and from how many 16-byte pieces on (16 x 4096 kept tokens
// of 8 heads of 128: 1, 2, 4 rows 39.5, 36.6, 38.1 us.  Whole calls in 1 and 2
// rows: 2^18 pieces 26.8 and 27.7, 2^20 40.9 and 39.9, 2^21 56.9 and 55.5).
constexpr int kRowsMany = 2;
constexpr int64_t kManyPieces = 1 << 19;

// Masses as integers of the same order; NaN below everything.
__device__ __forceinline__ uint32_t mass_key(float f)
{
    if (f != f)
        return 0;
    const uint32_t u = std::bit_cast<uint32_t>(f == 0.0f ? 0.0f : f);  // -0 is 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum over the workgroup's threads, in their order.
template <int WAVES>
__device__ __forceinline__ int block_before(int v, int *wsum)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(sum, d);
        sum += lane >= d ? o : 0;
    }
    if (lane == 63)
        wsum[wave] = sum;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i)
        before += i < wave ? wsum[i] : 0;
    return before + sum - v;
}

// One workgroup per (head, sequence).  Thread `tid` has the tokens per * tid ..
// + per - 1; HELD of them at most stay in registers as keys (HELD >= per), or,
// with HELD = 0, they are read again on every pass.
template <int SEL, int HELD>
__global__ __launch_bounds__(SEL) void kv_select_kernel(KvCache c, KvBatch b, const float *__restrict__ mass,
                                                         int64_t width, int budget, int recent,
                                                         int32_t *__restrict__ new_lens, float *__restrict__ new_mass,
                                                         int64_t new_width, int32_t *__restrict__ kept, int per)
{
    constexpr int WAVES = SEL / 64;
    __shared__ int counts[2][3][16], wsum[3][WAVES], gone[WAVES], first_recent;
    const int h = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int len = min(max(b.lens[seq], 0), b.max_len);
    const int64_t rowid = (int64_t)seq * c.heads + h;
    const float *m = mass + rowid * width;
    float *mo = new_mass + rowid * new_width;
    int32_t *ko = kept + rowid * budget;
    int n = min(len, budget), old = len - recent;  // tokens from `old` on are recent
    const int t0 = per * tid;
    // keys of the thread's tokens; 0, which no candidate value is, where there
    // is no old token.  Bit i of `here`: token i of the thread is there.
    uint32_t key[HELD ? HELD : 1], here = 0;
    if constexpr (HELD) {
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            key[i] = i < per && t0 + i < old ? mass_key(m[t0 + i]) : 0u;
        const int mine = min(max(len - t0, 0), per);
        here = mine >= 32 ? ~0u : (1u << mine) - 1;
    }
    // whether any page of the sequence is missing
    const int32_t *table = b.table + (int64_t)seq * b.table_width;
    bool miss = false;
    for (int p = tid; p < (len + (1 << c.page_shift) - 1) >> c.page_shift; p += SEL)
        miss = miss || (unsigned)table[p] >= (unsigned)c.pages;
    miss = __any(miss);
    if (lane == 0)
        gone[wave] = miss;
    __syncthreads();
    const bool holes = __any(gone[min(lane, WAVES - 1)] != 0);
    auto there = [&](int t) { return t < len && (!holes || (unsigned)table[t >> c.page_shift] < (unsigned)c.pages); };
    if (holes) {
        int mine = 0;
        for (int i = 0; i < per; ++i)
            mine += there(t0 + i);
        int rank = block_before<WAVES>(mine, wsum[2]), all = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            all += wsum[2][w];
        n = min(all, budget);
        if (tid == 0)
            first_recent = len;
        __syncthreads();
        // (all that are there stay where they do not exceed the budget)
        const int first = all <= budget ? 0 : all - recent;
        for (int i = 0; i < per; ++i)
            if (there(t0 + i) && rank++ == first)
                first_recent = t0 + i;
        __syncthreads();
        old = all <= budget ? 0 : first_recent;
        for (int i = n + tid; i < budget; i += SEL)
            ko[i] = -1;
        if constexpr (HELD) {
            for (int i = 0; i < per; ++i)
                if (!there(t0 + i))
                    here &= ~(1u << i);
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                key[i] = (here >> i & 1) && t0 + i < old ? mass_key(m[t0 + i]) : 0u;
        }
    }
    if (h == 0 && tid == 0)
        new_lens[seq] = n;
    for (int64_t i = n + tid; i < new_width; i += SEL)
        mo[i] = 0.0f;
    if (len <= budget && !holes) {
        for (int i = tid; i < n; i += SEL)
            mo[i] = m[i];
        for (int i = tid; i < budget; i += SEL)
            ko[i] = i < n ? i : -1;
        return;
    }
    const int want = old == 0 ? 0 : budget - recent;  // of the tokens before `old`, fewer than they are
    auto stands = [&](int i) -> bool {
        if constexpr (HELD)
            return here >> i & 1;
        else
            return there(t0 + i);
    };
    uint32_t T = 0;
    int above = 0;  // keys above T
    for (int shift = 30; shift >= 0; shift -= 2) {
        int cnt[3] = {0, 0, 0};
        auto count = [&](uint32_t k) {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                cnt[e] += __popcll(__ballot(k >= (T | (uint32_t)(e + 1) << shift)));
        };
        if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                count(key[i]);
        } else {
            // (in strides here: no order is needed to count)
            for (int t = tid; t < per * SEL; t += SEL)
                count(t < old && there(t) ? mass_key(m[t]) : 0u);
        }
        int(&to)[3][16] = counts[(shift >> 1) & 1];
        if (lane < 3)
            to[lane][wave] = lane == 0 ? cnt[0] : lane == 1 ? cnt[1] : cnt[2];
        __syncthreads();
        // the waves' counts of a candidate in 16 lanes, summed by rotations
        static_assert(WAVES <= 16, "a row of lanes a candidate");
        int all = lane < 48 && (lane & 15) < WAVES ? to[lane >> 4][lane & 15] : 0;
        all += __builtin_amdgcn_update_dpp(0, all, 0x128, 0xf, 0xf, true);
        all += __builtin_amdgcn_update_dpp(0, all, 0x124, 0xf, 0xf, true);
        all += __builtin_amdgcn_update_dpp(0, all, 0x122, 0xf, 0xf, true);
        all += __builtin_amdgcn_update_dpp(0, all, 0x121, 0xf, 0xf, true);
        const int sum[3] = {__builtin_amdgcn_readlane(all, 0), __builtin_amdgcn_readlane(all, 16),
                            __builtin_amdgcn_readlane(all, 32)};
        // sum[0] >= sum[1] >= sum[2]: the largest candidate that `want` reach
        const int d = sum[2] >= want ? 3 : sum[1] >= want ? 2 : sum[0] >= want ? 1 : 0;
        if (d < 3)
            above = sum[d];
        T |= (uint32_t)d << shift;
        // exactly `want` reach T: no later bit matters (without ties this
        // comes after about 24 of 32 bits)
        if (d > 0 && sum[max(d, 1) - 1] == want) {
            T -= 1;
            above = want;
            break;
        }
    }
    // `above` was last set where a digit was not 3: the keys past the prefix
    // T then had, which are those above T (later digits of 3 leave none between)
    const int need = want - above;  // tokens equal to T to take
    auto key_at = [&](int i) -> uint32_t {
        if constexpr (HELD)
            return key[i];
        else
            return t0 + i < old ? mass_key(m[t0 + i]) : 0u;
    };
    int ties = 0;
    auto each = [&](auto &&fn) {
        if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                if (i < per)
                    fn(i);
        } else {
            for (int i = 0; i < per; ++i)
                fn(i);
        }
    };
    each([&](int i) { ties += t0 + i < old && stands(i) && key_at(i) == T; });
    int tie = block_before<WAVES>(ties, wsum[0]);
    auto stays = [&](int i) -> bool {  // in order of i, once
        const int t = t0 + i;
        if (!stands(i))
            return false;
        if (t >= old)
            return true;
        const uint32_t k = key_at(i);
        return k > T || (k == T && tie++ < need);
    };
    // (the kept tokens' masses, asked for together before the places are known)
    float val[HELD ? HELD : 1];
    if constexpr (HELD) {
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            val[i] = i < per ? m[min(t0 + i, len - 1)] : 0.0f;
    }
    int stay = 0;
    const int tie0 = tie;
    each([&](int i) { stay += stays(i); });
    int place = block_before<WAVES>(stay, wsum[1]);
    tie = tie0;
    each([&](int i) {
        if (stays(i)) {
            ko[place] = t0 + i;
            mo[place] = HELD ? val[HELD ? i : 0] : m[t0 + i];
            ++place;
        }
    });
}

// N bytes of an array of N-byte rows, by the widest accesses that their
// alignment allows.
template <int N>
struct Bytes {
    uint32_t w[(N + 3) / 4];
    __device__ __forceinline__ void load(const uint8_t *from)
    {
        if constexpr (N % 16 == 0) {
#pragma unroll
            for (int i = 0; i < N / 16; ++i) {
                const u32x4 v = ((const u32x4 *)from)[i];
                w[4 * i] = v[0], w[4 * i + 1] = v[1], w[4 * i + 2] = v[2], w[4 * i + 3] = v[3];
            }
        } else if constexpr (N == 8) {
            const u32x2 v = *(const u32x2 *)from;
            w[0] = v[0], w[1] = v[1];
        } else if constexpr (N == 4) {
            w[0] = *(const uint32_t *)from;
        } else if constexpr (N == 2) {
            w[0] = *(const uint16_t *)from;
        } else {
            static_assert(N == 1, "rows of 1, 2, 4, 8 or a multiple of 16 bytes");
            w[0] = *from;
        }
    }
    __device__ __forceinline__ void store(uint8_t *to) const
    {
        if constexpr (N % 16 == 0) {
#pragma unroll
            for (int i = 0; i < N / 16; ++i)
                ((u32x4 *)to)[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        } else if constexpr (N == 8) {
            *(u32x2 *)to = u32x2{w[0], w[1]};
        } else if constexpr (N == 4) {
            *(uint32_t *)to = w[0];
        } else if constexpr (N == 2) {
            *(uint16_t *)to = (uint16_t)w[0];
        } else {
            *to = (uint8_t)w[0];
        }
    }
};

// SB: bytes of scales a row, ZB: of zero-points; U rows a lane, their loads
// (token, pages, row) in flight together.  A place without a token or a page
// reads row 0 of the pool and stores nothing.
template <int D, int SB, int ZB, int U>
__global__ __launch_bounds__(kMove) void kv_move_kernel(KvCache c, KvBatch b, const int32_t *__restrict__ new_table,
                                                        int new_tw, int budget, const int32_t *__restrict__ kept)
{
    constexpr int LANES = D / 32;  // 16 bytes of codes a lane
    const int h = blockIdx.y, seq = blockIdx.z;
    const int chunk = threadIdx.x % LANES;
    const int64_t place0 = ((int64_t)blockIdx.x * U * kMove + threadIdx.x) / LANES;
    const int32_t *from = kept + ((int64_t)seq * c.heads + h) * budget;
    const int32_t *table = b.table + (int64_t)seq * b.table_width, *ntable = new_table + (int64_t)seq * new_tw;
    int t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t place = place0 + u * (kMove / LANES);
        t[u] = from[min(place, (int64_t)budget - 1)];
        if (place >= budget)
            t[u] = -1;
    }
    int64_t src[U], dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int place = t[u] < 0 ? 0 : (int)(place0 + u * (kMove / LANES));
        src[u] = kv_row(c, table, max(t[u], 0), h);
        dst[u] = kv_row(c, ntable, place, h);
        if (t[u] < 0 || src[u] < 0)
            dst[u] = -1;
        src[u] = max(src[u], (int64_t)0);
    }
    const KvHalf &x = chunk & 1 ? c.v : c.k;  // whose scales the lane moves
    Bytes<16> k[U], v[U];
    Bytes<SB> sc[U];
    Bytes<ZB ? ZB : 1> z[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        k[u].load(c.k.codes + src[u] * (D / 2) + 16 * chunk);
        v[u].load(c.v.codes + src[u] * (D / 2) + 16 * chunk);
        if (chunk < 2) {
            sc[u].load((const uint8_t *)x.scales + src[u] * SB);
            if constexpr (ZB > 0)
                z[u].load(x.zeros + src[u] * ZB);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (dst[u] < 0)
            continue;
        k[u].store(c.k.codes + dst[u] * (D / 2) + 16 * chunk);
        v[u].store(c.v.codes + dst[u] * (D / 2) + 16 * chunk);
        if (chunk < 2) {
            sc[u].store((uint8_t *)x.scales + dst[u] * SB);
            if constexpr (ZB > 0)
                z[u].store(x.zeros + dst[u] * ZB);
        }
    }
}

template <int D, int SB, int ZB>
void move(const KvCache &c, const KvBatch &b, const int32_t *new_table, int new_tw, int budget, const int32_t *kept,
          hipStream_t s)
{
    const int64_t items = (int64_t)budget * (D / 32);
    auto go = [&](auto rows) {
        constexpr int U = decltype(rows)::value;
        const unsigned wgs = (unsigned)((items + U * kMove - 1) / (U * kMove));
        kv_move_kernel<D, SB, ZB, U><<<dim3(wgs, c.heads, b.seqs), kMove, 0, s>>>(c, b, new_table, new_tw, budget, kept);
    };
    items * c.heads * b.seqs >= kManyPieces ? go(KvInt<kRowsMany>{}) : go(KvInt<1>{});
}

}  // namespace

hipError_t launch_kv_evict(int f, const KvCache &c, const KvBatch &b, const float *mass,
                           int64_t mass_width, const int32_t *new_table, int new_table_width,
                           int budget, int recent, int32_t *new_lens, float *new_mass,
                           int64_t new_width, int32_t *kept, hipStream_t s)
{
    const dim3 grid(c.heads, b.seqs);
    // up to 4096 tokens in four waves (one to a SIMD: a pass over the candidates
    // is a few hundred cycles of latency, which more waves only lengthen), else
    // in sixteen (calls: 1088 tokens 13.2 and 16.7 us, 2048 13.3 and 16.8, 4096
    // 20.0 and 19.1)
    const int threads = b.max_len <= 16 * kSelFew ? kSelFew : kSel;
    const int per = std::max(1, (b.max_len + threads - 1) / threads);
    auto select = [&](auto sel, auto held) {
        constexpr int SEL = decltype(sel)::value;
        kv_select_kernel<SEL, decltype(held)::value><<<grid, SEL, 0, s>>>(c, b, mass, mass_width, budget, recent, new_lens,
                                                                          new_mass, new_width, kept, per);
    };
    if (threads == kSelFew)
        per <= 4   ? select(KvInt<kSelFew>{}, KvInt<4>{})
        : per <= 8 ? select(KvInt<kSelFew>{}, KvInt<8>{})
                   : select(KvInt<kSelFew>{}, KvInt<16>{});
    else if (per <= 8)
        select(KvInt<kSel>{}, KvInt<8>{});
    else if (per <= 16)
        select(KvInt<kSel>{}, KvInt<16>{});
    else if (per <= 32)
        select(KvInt<kSel>{}, KvInt<32>{});
    else
        select(KvInt<kSel>{}, KvInt<0>{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int sb = c.dim / c.g * (f32_absmax(f) ? 4 : 2), zb = f == Q4_INT4_ASYM ? kv_zero_bytes(c.dim, c.g) : 0;
    // every pair of scale and zero-point bytes that a format, width and group give
    auto go = [&](auto dim) -> hipError_t {
        constexpr int D = decltype(dim)::value;
        auto with = [&](auto s2, auto z2) {
            move<D, decltype(s2)::value, decltype(z2)::value>(c, b, new_table, new_table_width, budget, kept, s);
            return hipGetLastError();
        };
        switch (sb * 8 + zb) {
        case 2 * 8: return with(KvInt<2>{}, KvInt<0>{});
        case 2 * 8 + 1: return with(KvInt<2>{}, KvInt<1>{});
        case 4 * 8: return with(KvInt<4>{}, KvInt<0>{});
        case 4 * 8 + 1: return with(KvInt<4>{}, KvInt<1>{});
        case 8 * 8: return with(KvInt<8>{}, KvInt<0>{});
        case 8 * 8 + 2: return with(KvInt<8>{}, KvInt<2>{});
        case 16 * 8: return with(KvInt<16>{}, KvInt<0>{});
        case 16 * 8 + 4: return with(KvInt<16>{}, KvInt<4>{});
        case 32 * 8: return with(KvInt<32>{}, KvInt<0>{});
        }
        return hipErrorInvalidValue;
    };
    return c.dim == 64 ? go(KvInt<64>{}) : c.dim == 128 ? go(KvInt<128>{}) : go(KvInt<256>{});
}

}  // namespace q4
