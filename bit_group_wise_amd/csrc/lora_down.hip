// lora_down.hip -- the rows' products with the adapters' long sides, h[m] =
// s x[m] A^T and u[m] = s dy[m] B.
//
// Both contract a long axis (K or N, thousands) to at most 256 values a row,
// so they are bound by reading x (or dy), and with a few rows by reading the
// adapters.  A [rank, K] is read as it lies, 8 consecutive k a lane; B [N,
// rank] has the contraction in its rows and comes from LDS transposed
// (ds_read_b64_tr_b16, see gemm_dx_tile.hpp).  The matrix cores' first operand
// is the adapter (16 values r), the second 16 rows, so a result lane holds 4
// consecutive r of one row.  Rows of several adapters are done adapter by
// adapter; where rows are few the adapters are spread over workgroups.
//  * Few rows (q4_lora_gemm up to 96): 16 rows a workgroup of 4 waves, whose
//    waves alternate over the long axis' steps of 32 with the operands straight
//    in registers.  The axis is cut into parts on different workgroups, whose
//    binary32 sums the kernel that reads them adds in order (no atomics).
//  * More: 64 rows a workgroup, both operands staged in LDS 64 of the axis at a
//    time, so that a row's lines are read whole and the adapter's matrix once
//    for 64 rows: what a compute unit can load (20 to 40 bytes a cycle) is the
//    limit, and with 16 rows a workgroup half of it was the adapter's matrix
//    (25 and 40 us on 2048 rows of 4096 with rank 32 and of 11008 with rank 16).
//    The axis' parts are joined by a second launch, which also splits the sums
//    into the three bfloat16 operands that their readers need.  (Readers that add
//    up 8 parts spent 20 to 130 us on it, one latency after another.)
#include "lora.hpp"
#include "q4_internal.hpp"

namespace q4 {
namespace {

// Four values r of row m as their operands, at split[(3 m + i) * rank + r].
__device__ __forceinline__ void store_split(uint16_t *split, int rank, int64_t m, int r, const f32x4 &v)
{
    const Split3 a = split3(v[0], v[1]), b = split3(v[2], v[3]);
    uint16_t *to = split + 3 * m * rank + r;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        *(u32x2 *)(to + i * rank) = u32x2{a.p[i], b.p[i]};
}

// ---------------------------------------------------------------- few rows
constexpr int kFewWaves = 4, kFewBlock = 64 * kFewWaves;

// One step's operands: 32 of the long axis for the adapter (8 consecutive
// values of a row r a lane) and for the rows.
template <int RF>
struct FewStep {
    u32x4 w[RF];
    u32x4 x;
};

// blockIdx: x the rows, y the part of the long axis, z slices of r and
// adapters' slots.
template <int ACT, int RF>
__global__ __launch_bounds__(kFewBlock) void down_few_kernel(DownArgs a)
{
    __shared__ f32x4 red[kFewWaves][RF][64];
    const int lane = threadIdx.x & 63;
    const int wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fi = lane & 15, fq = lane >> 4;
    const int slice = blockIdx.z % a.slices, slot = blockIdx.z / a.slices;
    const int len = a.K, r0 = slice * 16 * RF;
    const int64_t m0 = (int64_t)blockIdx.x * 16;
    const int rows = (int)(a.rows - m0 < 16 ? a.rows - m0 : 16);
    const __amdgpu_buffer_rsrc_t xr = buffer_view((const uint16_t *)a.x + m0 * len, (int64_t)rows * len * 2);
    // this part's steps of 32
    const int steps = (len + 31) / 32, per = (steps + a.parts - 1) / a.parts;
    const int first = blockIdx.y * per, last = min(first + per, steps);

    AdapterSet<1> set;
    set.init(a.ids, a.adapters, m0, rows);
    int ad, at = 0;
    uint64_t mask[1];
    while (set.next(ad, mask)) {
        if (at++ % a.slots != slot)
            continue;
        const __amdgpu_buffer_rsrc_t wr =
            buffer_view((const uint16_t *)a.a + (int64_t)ad * a.rank * len, (int64_t)a.rank * len * 2);
        auto load = [&](FewStep<RF> &st, int step) {
            const int k = 32 * step + 8 * fq;
            const bool on = step < last && k < len;
#pragma unroll
            for (int f = 0; f < RF; ++f) {
                const int r = r0 + 16 * f + fi;
                st.w[f] = __builtin_amdgcn_raw_buffer_load_b128(wr, on && r < a.rank ? 2 * (r * len + k) : -16, 0, 0);
            }
            st.x = __builtin_amdgcn_raw_buffer_load_b128(xr, on && fi < rows ? 2 * (fi * len + k) : -16, 0, 0);
        };
        f32x4 acc[RF];
#pragma unroll
        for (int f = 0; f < RF; ++f)
            acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        constexpr int kRing = 4;
        FewStep<RF> ring[kRing];
#pragma unroll
        for (int i = 0; i < kRing; ++i)
            load(ring[i], first + wave + kFewWaves * i);
        for (int step = first + wave; step < last; step += kFewWaves * kRing) {
#pragma unroll
            for (int i = 0; i < kRing; ++i) {
#pragma unroll
                for (int f = 0; f < RF; ++f)
                    acc[f] = mfma<ACT>(ring[i].w[f], ring[i].x, acc[f]);
                load(ring[i], step + kFewWaves * (i + kRing));
            }
        }
        __syncthreads();  // (the last adapter's sums have been read)
#pragma unroll
        for (int f = 0; f < RF; ++f)
            red[wave][f][lane] = acc[f];
        __syncthreads();
        const float s = a.scale ? a.scale[ad] : 1.0f;
        for (int f = wave; f < RF; f += kFewWaves) {
            f32x4 v = red[0][f][lane];
#pragma unroll
            for (int i = 1; i < kFewWaves; ++i) {
                const f32x4 u = red[i][f][lane];
                v = f32x4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
            }
            const int r = r0 + 16 * f + 4 * fq;
            if (((rows16(mask[0], 0) >> fi) & 1) && r < a.rank)
                *(f32x4 *)((float *)a.h + (blockIdx.y * a.rows + m0 + fi) * a.rank + r) =
                    f32x4{v[0] * s, v[1] * s, v[2] * s, v[3] * s};
        }
    }
}

// --------------------------------------------------------------- more rows
constexpr int kBlock = 256;  // 4 waves of 16 rows
constexpr int kRows = kDownRows;
constexpr int kStep = kDownStep;  // of the long axis
constexpr int kAhead = 3;    // steps whose loads are in flight in registers

// Position of 16-byte chunk c of a staged row of 128 bytes.
__device__ __forceinline__ int dswz(int r, int c) { return c ^ ((r >> 1) & 7); }
// Byte offset of chunk c (8 values r) of staged row n of B (32 RF bytes a row):
// pairs of chunks, which a transposed read takes together, are exchanged so
// that its 4 rows and the next lanes' 4, 8 rows on, lie in other banks.
template <int RF>
__device__ __forceinline__ int bofs(int n, int c)
{
    constexpr int pairs = RF;
    const int key = pairs == 4 ? (n & 3) ^ ((n >> 3) & 1) : (pairs == 2 ? (n >> 3) & 1 : 0);
    return n * 32 * RF + 16 * (c ^ (2 * key));
}

// A thread's loads of a step: x's 16-byte chunks t % 8 of rows t / 8 + 32 i,
// and the adapter's: of A as x's, of B chunks of its 64 rows one after another.
template <int RF>
struct ManyStep {
    u32x4 x[2];
    u32x4 w[RF > 2 ? 2 : 1];
};

template <int ACT, int RF, bool TRANS>
__device__ __forceinline__ void down_many(const DownArgs &a, const uint16_t *__restrict__ x,
                                          const uint16_t *__restrict__ w, uint16_t *split, float *part, int len,
                                          int slice, int slot, char (&xs)[2][kRows * 128], char (&ws)[2][RF * 2048])
{
    constexpr int kW = RF > 2 ? 2 : 1;  // loads of the adapter a thread
    const int t = threadIdx.x, lane = t & 63;
    const int wave = (int)__builtin_amdgcn_readfirstlane(t >> 6);
    const int fi = lane & 15, fq = lane >> 4;
    const int r0 = slice * 16 * RF;
    const int64_t m0 = (int64_t)blockIdx.x * kRows;
    const int rows = (int)(a.rows - m0 < kRows ? a.rows - m0 : kRows);
    const __amdgpu_buffer_rsrc_t xr = buffer_view(x + m0 * len, (int64_t)rows * len * 2);
    const int steps = (len + kStep - 1) / kStep, per = (steps + a.parts - 1) / a.parts;
    const int first = blockIdx.y * per, last = min(first + per, steps);

    AdapterSet<1> set;
    set.init(a.ids, a.adapters, m0, rows);
    int ad, at = 0;
    uint64_t mask[1];
    while (set.next(ad, mask)) {
        if (at++ % a.slots != slot)
            continue;
        const __amdgpu_buffer_rsrc_t wr = buffer_view(w + (int64_t)ad * a.rank * len, (int64_t)a.rank * len * 2);
        auto load = [&](ManyStep<RF> &st, int step) {
            const int k = kStep * step + 8 * (t & 7);
            const bool on = step < last;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int m = (t >> 3) + 32 * i;
                st.x[i] = __builtin_amdgcn_raw_buffer_load_b128(
                    xr, on && k < len && m < rows ? 2 * (m * len + k) : -16, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                int off = -16;
                if constexpr (TRANS) {
                    const int p = t + kBlock * i, n = kStep * step + p / (2 * RF), r = r0 + 8 * (p % (2 * RF));
                    if (on && p < 128 * RF && n < len && r < a.rank)
                        off = 2 * (n * a.rank + r);
                } else {
                    const int r = r0 + (t >> 3) + 32 * i;
                    if (on && k < len && (t >> 3) + 32 * i < 16 * RF && r < a.rank)
                        off = 2 * (r * len + k);
                }
                st.w[i] = __builtin_amdgcn_raw_buffer_load_b128(wr, off, 0, 0);
            }
        };
        auto store = [&](const ManyStep<RF> &st, char *xb, char *wb) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int m = (t >> 3) + 32 * i;
                *(u32x4 *)(xb + m * 128 + 16 * dswz(m, t & 7)) = st.x[i];
            }
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                if constexpr (TRANS) {
                    const int p = t + kBlock * i;
                    if (p < 128 * RF)
                        *(u32x4 *)(wb + bofs<RF>(p / (2 * RF), p % (2 * RF))) = st.w[i];
                } else {
                    const int r = (t >> 3) + 32 * i;
                    if (r < 16 * RF)
                        *(u32x4 *)(wb + r * 128 + 16 * dswz(r, t & 7)) = st.w[i];
                }
            }
        };
        f32x4 acc[RF];
#pragma unroll
        for (int f = 0; f < RF; ++f)
            acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        auto work = [&](const char *xb, const char *wb) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = 16 * wave + fi;
                const u32x4 xf = *(const u32x4 *)(xb + m * 128 + 16 * dswz(m, 4 * h + fq));
#pragma unroll
                for (int f = 0; f < RF; ++f) {
                    u32x4 wf;
                    if constexpr (TRANS) {
                        const auto at = [&](int u) {
                            return wb + bofs<RF>(32 * h + 8 * fq + 4 * u + (fi >> 2), 2 * f + ((fi >> 1) & 1)) + 8 * (fi & 1);
                        };
                        wf = read_column8(at(0), at(1));
                    } else {
                        const int r = 16 * f + fi;
                        wf = *(const u32x4 *)(wb + r * 128 + 16 * dswz(r, 4 * h + fq));
                    }
                    acc[f] = mfma<ACT>(wf, xf, acc[f]);
                }
            }
        };
        // steps in flight in registers, the current one in one of two LDS
        // buffers: one barrier a step (whoever writes a buffer has passed the
        // barrier behind the reads of its last contents)
        ManyStep<RF> ring[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            load(ring[i], first + i);
        __syncthreads();  // (the last adapter's tiles have been read)
        for (int step = first; step < last; step += 2 * kAhead) {
#pragma unroll
            for (int i = 0; i < 2 * kAhead; ++i) {
                if (step + i >= last)
                    break;
                store(ring[i % kAhead], xs[i & 1], ws[i & 1]);
                load(ring[i % kAhead], step + i + kAhead);
                __syncthreads();
                work(xs[i & 1], ws[i & 1]);
            }
        }
        const float s = a.scale ? a.scale[ad] : 1.0f;
        const bool mine = (rows16(mask[0], 16 * wave) >> fi) & 1;
#pragma unroll
        for (int f = 0; f < RF; ++f) {
            const int r = r0 + 16 * f + 4 * fq;
            if (!mine || r >= a.rank)
                continue;
            const f32x4 v{acc[f][0] * s, acc[f][1] * s, acc[f][2] * s, acc[f][3] * s};
            const int64_t m = m0 + 16 * wave + fi;
            if (a.parts > 1)
                *(f32x4 *)(part + (blockIdx.y * a.rows + m) * a.rank + r) = v;
            else
                store_split(split, a.rank, m, r, v);
        }
    }
}

// blockIdx: x the rows, y the part of the long axis, z slices of r, adapters'
// slots and (h, u) where both are wanted.
template <int ACT, int RF>
__global__ __launch_bounds__(kBlock) void down_many_kernel(DownArgs a)
{
    __shared__ __attribute__((aligned(16))) char xs[2][kRows * 128];
    __shared__ __attribute__((aligned(16))) char ws[2][RF * 2048];
    int z = blockIdx.z;
    const int slice = z % a.slices;
    z /= a.slices;
    const int slot = z % a.slots;
    z /= a.slots;
    if (a.x && z == 0)
        down_many<ACT, RF, false>(a, (const uint16_t *)a.x, (const uint16_t *)a.a, (uint16_t *)a.h, a.sums, a.K, slice,
                                  slot, xs, ws);
    else
        down_many<ACT, RF, true>(a, (const uint16_t *)a.dy, (const uint16_t *)a.b, (uint16_t *)a.u,
                                 a.sums + (a.x ? a.parts * a.rows * a.rank : 0), a.N, slice, slot, xs, ws);
}

// The parts' sums added in order and split into operands, 4 values a thread
// (rank is a multiple of 8); blockIdx.y: h, u.
__global__ __launch_bounds__(256) void down_join_kernel(DownArgs a)
{
    const int64_t size = a.rows * a.rank, at = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (at >= size)
        return;
    const bool h = a.x && blockIdx.y == 0;
    const float *p = a.sums + (blockIdx.y ? a.parts * size : 0) + at;
    f32x4 v = *(const f32x4 *)p;
#pragma unroll
    for (int i = 1; i < kMostParts; ++i) {
        if (i < a.parts) {
            const f32x4 u = *(const f32x4 *)(p + i * size);
            v = f32x4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
        }
    }
    const int64_t m = at / a.rank;
    store_split((uint16_t *)(h ? a.h : a.u), a.rank, m, (int)(at - m * a.rank), v);
}

template <int ACT>
hipError_t launch_dn(const DownArgs &a, const DownPlan &p, hipStream_t s)
{
    const int kinds = (a.x ? 1 : 0) + (a.dy ? 1 : 0);
    const dim3 grid((unsigned)p.tiles, (unsigned)a.parts, (unsigned)(a.slices * a.slots * kinds));
    if (!p.split) {
        if (p.rf == 1)
            hipLaunchKernelGGL((down_few_kernel<ACT, 1>), grid, dim3(kFewBlock), 0, s, a);
        else if (p.rf == 2)
            hipLaunchKernelGGL((down_few_kernel<ACT, 2>), grid, dim3(kFewBlock), 0, s, a);
        else
            hipLaunchKernelGGL((down_few_kernel<ACT, 4>), grid, dim3(kFewBlock), 0, s, a);
        return hipGetLastError();
    }
    if (p.rf == 1)
        hipLaunchKernelGGL((down_many_kernel<ACT, 1>), grid, dim3(kBlock), 0, s, a);
    else if (p.rf == 2)
        hipLaunchKernelGGL((down_many_kernel<ACT, 2>), grid, dim3(kBlock), 0, s, a);
    else
        hipLaunchKernelGGL((down_many_kernel<ACT, 4>), grid, dim3(kBlock), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1)
        return e;
    const dim3 joins((unsigned)((a.rows * a.rank / 4 + 255) / 256), (unsigned)kinds);
    hipLaunchKernelGGL(down_join_kernel, joins, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_down(q4_dtype act_t, DownArgs a, const DownPlan &p, hipStream_t s)
{
    a.slices = p.slices;
    a.slots = p.slots;
    a.parts = p.parts;
    return act_t == Q4_BF16 ? launch_dn<Q4_BF16>(a, p, s) : launch_dn<Q4_F16>(a, p, s);
}

}  // namespace q4
