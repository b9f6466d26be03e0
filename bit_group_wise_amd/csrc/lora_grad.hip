// lora_grad.hip -- the adapters' gradients, dA[a] = sum_m u[m]^T x[m] and
// dB[a] = sum_m dy[m]^T h[m] over the rows m of adapter a.
//
// Both are G[c][r] = sum_m X[m][c] P[m][r] with a short side r (P = u or h)
// and a long one c (X = x or dy), so they are bound by reading X once.  A
// workgroup of 4 waves takes 128 columns c, up to 64 values r and one part of
// the rows, 64 rows a step:
//  * the contraction runs over the rows, so both operands need 8 consecutive
//    rows of one column: X's 64 x 128 tile and P's (its three bfloat16 parts side
//    by side; of 64 values r the third in a tile of its own) lie in LDS row by
//    row and come back transposed (ds_read_b64_tr_b16; layout and bank spread as
//    in gemm_dx_tile.hpp);
//  * rows of other adapters enter both tiles as zeros, and steps without a row
//    of this adapter are left out: the rows' adapters are looked through first,
//    256 steps at a time;
//  * the loads of the next three steps are in flight while one's products run
//    (with one, 8 steps a workgroup took 29 us where the rows' bytes take 13);
//  * dA's accumulators hold columns in a lane and dB's values r, so each is
//    stored along its own rows;
//  * with few columns and adapters the rows are split over workgroups, whose
//    binary32 sums a second kernel adds in order and rounds.
#include "lora.hpp"
#include "q4_internal.hpp"

namespace q4 {
namespace {

constexpr int kGrWaves = 4;
constexpr int kGrBlock = 64 * kGrWaves;
constexpr int kGrPitch = 288;   // bytes of a staged row of 128 values
constexpr int kGrList = 256;    // steps listed at a time

__device__ __forceinline__ int gofs(int row, int col) { return row * kGrPitch + ((2 * col) ^ (((row >> 3) & 1) << 7)); }

// 8 rows of one column as an operand: rows 32 h + 8 fq .. + 7, column c0 + fi.
__device__ __forceinline__ u32x4 column8(const char *tile, int h, int c0)
{
    const int lane = threadIdx.x & 63, fi = lane & 15, fq = lane >> 4;
    const auto at = [&](int u) { return tile + gofs(32 * h + 8 * fq + 4 * u + (fi >> 2), c0 + 4 * (fi & 3)); };
    return read_column8(at(0), at(1));
}

// One kind of gradient: X [rows, cols], P's parts [rows, 3, rank], and the
// output [ad, rank, cols] (dA) or [ad, cols, rank] (dB).
struct Side {
    const uint16_t *x;
    const uint16_t *p;
    int cols;
    int64_t out;  // where the side's sums begin in a part of `sums`
    uint16_t *g;
};

// A thread's loads of a step: X's 16-byte chunks t % 16 of rows t / 16 + 16 i,
// and of each of P's parts 16-byte chunks one after another.
template <int RF>
struct GradStep {
    u32x4 x[4];
    u32x4 p[3][RF > 2 ? 2 : 1];
};

// Buffers of P, and of X with its parts: two, but of 64 values r one of P, and
// beside fp16 one of X, so that two workgroups still share a compute unit's LDS
// (67 KB each).  The backward pass of 4096 rows through 4096 x 4096 in us, two
// buffers and a workgroup a unit / this: rank 64 bfloat16 212 / 206, fp16 236 /
// 224; rank 128 241 / 234, 284 / 261.  (One of each for 16 or 32 values r of fp16:
// 283.6 / 284.5 on 2048 rows of 4096 x 11008, rank 16; 67.7 / 68.2 on 300 of 4096 x
// 4096, rank 32.)
template <int RF>
constexpr int kPBufs = RF > 2 ? 1 : 2;
template <int ACT, int RF>
constexpr int kXBufs = RF > 2 && ACT == Q4_F16 ? 1 : 2;

// The LDS of a workgroup: one or two steps' tiles, and the steps listed.  P's
// part i of value r lies in column PW i + r of its row; of 64 values the third,
// which has no room there, in column 64 (row / 32) + r of row % 32 of a tile of
// its own.
template <int ACT, int RF>
struct GradLds {
    char x[kXBufs<ACT, RF>][kGrRows * kGrPitch];
    char xlo[kXBufs<ACT, RF>][ACT == Q4_F16 ? kGrRows * kGrPitch : 16];
    char p[kPBufs<RF>][kGrRows * kGrPitch];
    char p2[RF > 2 ? kPBufs<RF> : 1][RF > 2 ? kGrRows / 2 * kGrPitch : 16];
    uint64_t mask[kGrList];  // rows of the adapter in the step
    uint16_t list[kGrList];
    int count;
};

template <int ACT, int RF, bool IS_B>
__device__ __forceinline__ void grad(const GradArgs &a, const Side &side, int cblock, int slice, int ad, int split,
                                     GradLds<ACT, RF> &lds)
{
    constexpr int PW = RF > 2 ? 64 : 32;        // columns a part
    constexpr bool kOneP = kPBufs<RF> == 1, kOneX = kXBufs<ACT, RF> == 1;
    constexpr int kPPieces = kGrRows * 2 * RF;  // 8-value pieces of P's tile
    constexpr int kPLoads = RF > 2 ? 2 : 1;     // ... a thread
    static_assert(kPPieces <= kPLoads * kGrBlock, "pieces of P");
    constexpr int kAhead = 3;                   // steps whose loads are in flight
    constexpr uint32_t kPast = 0x80000000u;     // past every view

    const int t = threadIdx.x, lane = t & 63;
    const int wave = (int)__builtin_amdgcn_readfirstlane(t >> 6);
    const int fi = lane & 15, fq = lane >> 4;
    const int c0 = cblock * kGrCols, r0 = slice * 16 * RF;
    const int64_t steps = (a.rows + kGrRows - 1) / kGrRows;
    const int64_t per = (steps + a.splits - 1) / a.splits;
    const int64_t first = split * per, last = first + per < steps ? first + per : steps;

    f32x4 acc[RF][2];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            acc[f][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int64_t base = first; base < last; base += kGrList) {
        // the steps with rows of this adapter, in order
        const int n = (int)(last - base < kGrList ? last - base : kGrList);
        __syncthreads();  // (the last list and tiles have been read)
        for (int s = wave; s < n; s += kGrWaves) {
            const int64_t m = (base + s) * kGrRows + lane;
            const uint64_t mine = __ballot(m < a.rows && adapter_of(a.ids, a.adapters, m < a.rows ? m : 0) == ad);
            if (lane == 0)
                lds.mask[s] = mine;
        }
        __syncthreads();
        if (wave == 0) {
            int found = 0;
            for (int s = 0; s < n; s += 64) {
                const bool on = s + lane < n && lds.mask[s + lane] != 0;
                const uint64_t m = __ballot(on);
                if (on)
                    lds.list[found + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0))] =
                        (uint16_t)(s + lane);
                found += __popcll(m);
            }
            if (lane == 0)
                lds.count = found;
        }
        __syncthreads();
        const int found = __builtin_amdgcn_readfirstlane(lds.count);

        // (rows of other adapters, past the end, and columns and values past
        // theirs are sent past the views and read as zeros; so are steps past
        // the last listed one)
        auto load = [&](GradStep<RF> &st, int i) {
            const bool on = i < found;
            const int s = __builtin_amdgcn_readfirstlane(on ? lds.list[i] : 0);
            const uint64_t mask = on ? lds.mask[s] : 0;
            const uint32_t halves[2] = {(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)mask),
                                        (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(mask >> 32))};
            const int64_t m0 = (base + s) * kGrRows;
            const int rows = (int)(a.rows - m0 < kGrRows ? a.rows - m0 : kGrRows);
            const __amdgpu_buffer_rsrc_t xr = buffer_view(side.x + m0 * side.cols, (int64_t)rows * side.cols * 2);
            const __amdgpu_buffer_rsrc_t pr = buffer_view(side.p + 3 * m0 * a.rank, (int64_t)rows * 3 * a.rank * 2);
            const int c = c0 + 8 * (t & 15);
            const uint32_t cpast = c < side.cols ? 0u : kPast;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = (t >> 4) + 16 * q;
                const uint32_t none = (halves[q / 2] >> (row & 31)) & 1 ? 0u : kPast;
                st.x[q] = __builtin_amdgcn_raw_buffer_load_b128(
                    xr, (int)(2u * (uint32_t)(row * side.cols + c) | none | cpast), 0, 0);
            }
#pragma unroll
            for (int q = 0; q < kPLoads; ++q) {
                const int p = t + kGrBlock * q, row = (p / (2 * RF)) & 63, r = r0 + 8 * (p % (2 * RF));
                const uint32_t its = halves[((64 * wave + kGrBlock * q) / (2 * RF)) >> 5 & 1];  // (a wave's rows lie in one)
                const uint32_t none = ((its >> (row & 31)) & 1) && p < kPPieces && r < a.rank ? 0u : kPast;
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    st.p[i][q] = __builtin_amdgcn_raw_buffer_load_b128(
                        pr, (int)(2u * (uint32_t)((3 * row + i) * a.rank + r) | none), 0, 0);
            }
        };
        auto store_x = [&](const GradStep<RF> &st, int buf) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const Exact8 w = exact_parts<ACT>(st.x[q]);
                const int at = gofs((t >> 4) + 16 * q, 8 * (t & 15));
                *(u32x4 *)(lds.x[buf] + at) = w.hi;
                if constexpr (ACT == Q4_F16)
                    *(u32x4 *)(lds.xlo[buf] + at) = w.lo;
            }
        };
        auto store_p = [&](const GradStep<RF> &st, int buf) {
#pragma unroll
            for (int q = 0; q < kPLoads; ++q) {
                const int p = t + kGrBlock * q;
                if (p < kPPieces) {
                    const int row = p / (2 * RF), r = 8 * (p % (2 * RF));
                    *(u32x4 *)(lds.p[buf] + gofs(row, r)) = st.p[0][q];
                    *(u32x4 *)(lds.p[buf] + gofs(row, PW + r)) = st.p[1][q];
                    if constexpr (RF > 2)
                        *(u32x4 *)(lds.p2[buf] + gofs(row & 31, 64 * (row >> 5) + r)) = st.p[2][q];
                    else
                        *(u32x4 *)(lds.p[buf] + gofs(row, 2 * PW + r)) = st.p[2][q];
                }
            }
        };
        auto work = [&](int buf, int pbuf) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Exact8 x[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    x[j].hi = column8(lds.x[buf], h, 32 * wave + 16 * j);
                    if constexpr (ACT == Q4_F16)
                        x[j].lo = column8(lds.xlo[buf], h, 32 * wave + 16 * j);
                }
#pragma unroll
                for (int f = 0; f < RF; ++f) {
                    const Low8 p{{column8(lds.p[pbuf], h, 16 * f), column8(lds.p[pbuf], h, PW + 16 * f),
                                  RF > 2 ? column8(lds.p2[pbuf], 0, 64 * h + 16 * f)
                                         : column8(lds.p[pbuf], h, 2 * PW + 16 * f)}};
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[f][j] = IS_B ? mfma_low_exact<ACT>(p, x[j], acc[f][j]) : mfma_exact_low<ACT>(x[j], p, acc[f][j]);
                }
            }
        };
        // steps in flight in registers, the current one in one of two LDS
        // buffers: one barrier a step, a second where there is one buffer
        GradStep<RF> ring[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            load(ring[i], i);
        for (int i0 = 0; i0 < found; i0 += 2 * kAhead) {
#pragma unroll
            for (int i = 0; i < 2 * kAhead; ++i) {
                if (i0 + i >= found)
                    break;
                if constexpr (kOneX)
                    __syncthreads();  // (the last step's tiles have been read)
                store_x(ring[i % kAhead], kOneX ? 0 : i & 1);
                if constexpr (kOneP && !kOneX)
                    __syncthreads();  // (the last step's P has been read)
                store_p(ring[i % kAhead], kOneP ? 0 : i & 1);
                load(ring[i % kAhead], i0 + i + kAhead);
                __syncthreads();
                work(kOneX ? 0 : i & 1, kOneP ? 0 : i & 1);
            }
        }
    }

    // dA: a lane has value r = fi of columns 4 fq ..; dB: column fi, values 4 fq ..
#pragma unroll
    for (int f = 0; f < RF; ++f) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int cb = c0 + 32 * wave + 16 * j;
            const int r = r0 + 16 * f + (IS_B ? 4 * fq : fi), c = cb + (IS_B ? fi : 4 * fq);
            if (r >= a.rank || c >= side.cols)
                continue;
            const int64_t at = IS_B ? ((int64_t)ad * side.cols + c) * a.rank + r : ((int64_t)ad * a.rank + r) * side.cols + c;
            const f32x4 v = acc[f][j];
            if (a.splits > 1)
                *(f32x4 *)(a.sums + (int64_t)split * a.adapters * a.rank * ((int64_t)a.N + a.K) + side.out + at) = v;
            else
                *(u32x2 *)(side.g + at) = u32x2{pack2<ACT>(v[0], v[1]), pack2<ACT>(v[2], v[3])};
        }
    }
}

// blockIdx: x columns of x, then of dy; y adapters and slices of r; z parts of the rows.
template <int ACT, int RF>
__global__ __launch_bounds__(kGrBlock, 2) void grad_kernel(GradArgs a, int slices)
{
    __shared__ __attribute__((aligned(16))) GradLds<ACT, RF> lds;
    const int kblocks = (a.K + kGrCols - 1) / kGrCols;
    const int slice = blockIdx.y % slices, ad = blockIdx.y / slices;
    const int64_t asize = (int64_t)a.adapters * a.rank * a.K;
    if ((int)blockIdx.x < kblocks) {
        const Side side{(const uint16_t *)a.x, a.u, a.K, 0, (uint16_t *)a.da};
        grad<ACT, RF, false>(a, side, blockIdx.x, slice, ad, blockIdx.z, lds);
    } else {
        const Side side{(const uint16_t *)a.dy, a.h, a.N, asize, (uint16_t *)a.db};
        grad<ACT, RF, true>(a, side, blockIdx.x - kblocks, slice, ad, blockIdx.z, lds);
    }
}

// The parts' sums added in order and rounded: 4 values a thread (both outputs
// are a multiple of 8 long).
template <int ACT>
__global__ __launch_bounds__(256) void grad_join_kernel(GradArgs a)
{
    const int64_t asize = (int64_t)a.adapters * a.rank * a.K, size = asize + (int64_t)a.adapters * a.rank * a.N;
    const int64_t at = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (at >= size)
        return;
    f32x4 v = *(const f32x4 *)(a.sums + at);
    for (int i = 1; i < a.splits; ++i) {
        const f32x4 u = *(const f32x4 *)(a.sums + i * size + at);
        v = f32x4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
    }
    uint16_t *to = at < asize ? (uint16_t *)a.da + at : (uint16_t *)a.db + (at - asize);
    *(u32x2 *)to = u32x2{pack2<ACT>(v[0], v[1]), pack2<ACT>(v[2], v[3])};
}

template <int ACT>
hipError_t launch_grad_act(const GradArgs &a, hipStream_t s)
{
    const int rf = grad_rf(a.rank), slices = (a.rank + 16 * rf - 1) / (16 * rf);
    const dim3 grid((unsigned)((a.K + kGrCols - 1) / kGrCols + (a.N + kGrCols - 1) / kGrCols),
                    (unsigned)(a.adapters * slices), (unsigned)a.splits);
    if (rf == 1)
        hipLaunchKernelGGL((grad_kernel<ACT, 1>), grid, dim3(kGrBlock), 0, s, a, slices);
    else if (rf == 2)
        hipLaunchKernelGGL((grad_kernel<ACT, 2>), grid, dim3(kGrBlock), 0, s, a, slices);
    else
        hipLaunchKernelGGL((grad_kernel<ACT, 4>), grid, dim3(kGrBlock), 0, s, a, slices);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1)
        return e;
    const int64_t size = (int64_t)a.adapters * a.rank * ((int64_t)a.K + a.N);
    hipLaunchKernelGGL((grad_join_kernel<ACT>), dim3((unsigned)((size / 4 + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_grad(q4_dtype act_t, const GradArgs &a, hipStream_t s)
{
    return act_t == Q4_BF16 ? launch_grad_act<Q4_BF16>(a, s) : launch_grad_act<Q4_F16>(a, s);
}

}  // namespace q4
