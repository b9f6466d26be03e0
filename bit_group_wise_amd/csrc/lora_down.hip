// lora_down.hip -- the rows' products with the adapters' long sides, h[m] =
// s x[m] A^T and u[m] = s dy[m] B, as binary32 partial sums.
//
// Both contract a long axis (K or N, thousands) to at most 256 values a row,
// so they are bound by reading x (or dy), and with a few rows by reading the
// adapters.  A workgroup of 4 waves takes 16 MT rows, up to 16 RF values r and
// one part of the long axis, over whose steps its waves alternate; their sums
// meet in LDS, and the parts in the kernel that reads them (which adds them in
// order: no atomics).
//  * The matrix cores' first operand is the adapter (16 values r), the second
//    16 rows, so a result lane holds 4 consecutive r of one row.
//  * A [rank, K] is read as it lies, 8 consecutive k a lane.  B [N, rank] has
//    the contraction in its rows: a wave stages 32 rows in its own LDS and
//    takes them back transposed (ds_read_b64_tr_b16, see gemm_dx_tile.hpp).
//  * Rows of several adapters are done adapter by adapter; where rows are few
//    the adapters of a tile are spread over workgroups.
#include "lora.hpp"
#include "q4_internal.hpp"

namespace q4 {
namespace {

constexpr int kDnWaves = 4;
constexpr int kDnBlock = 64 * kDnWaves;

typedef short v4i16 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t dn_rsrc(const void *base, int64_t bytes)
{
    const uint32_t n = __builtin_amdgcn_readfirstlane(
        bytes <= 0 ? 0u : (bytes >= 0x7fffffffll ? 0x7fffffffu : (uint32_t)bytes));
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)n, 0x00020000);
}

// One step's operands: 32 of the long axis for the adapter (as read: of A 8
// consecutive values of a row r a lane; of B 16-byte pieces of its rows) and
// for the rows.
template <int RF, int MT>
struct DnStep {
    u32x4 w[RF];
    u32x4 x[MT];
};

// Bytes of a staged row of B (not a multiple of 64: rows spread over the banks).
constexpr int dn_pitch(int rf) { return 32 * rf + 16; }

template <int ACT, int RF, int MT, bool TRANS>
__device__ __forceinline__ void down(const uint16_t *__restrict__ x, const DownArgs &a, const uint16_t *__restrict__ w,
                                     float *__restrict__ part, int len, int slice, int slot, int split,
                                     f32x4 (&red)[kDnWaves][RF][MT][64], char *stages)
{
    constexpr int kPitch = dn_pitch(RF);
    const int lane = threadIdx.x & 63;
    const int wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fi = lane & 15, fq = lane >> 4;
    char *stage = stages + wave * 32 * kPitch;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * MT);
    const int rows = (int)(a.rows - m0 < 16 * MT ? a.rows - m0 : 16 * MT);
    const int r0 = slice * 16 * RF;
    const __amdgpu_buffer_rsrc_t xr = dn_rsrc(x + m0 * len, (int64_t)rows * len * 2);
    // this part's steps of 32
    const int steps = (len + 31) / 32;
    const int per = (steps + a.parts - 1) / a.parts;
    const int first = split * per, last = min(first + per, steps);

    AdapterSet<1> set;
    set.init(a.ids, a.adapters, m0, rows);
    int ad, at = 0;
    uint64_t mask[1];
    while (set.next(ad, mask)) {
        if (at++ % a.slots != slot)
            continue;
        const __amdgpu_buffer_rsrc_t wr = dn_rsrc(w + (int64_t)ad * a.rank * len, (int64_t)a.rank * len * 2);
        auto load = [&](DnStep<RF, MT> &st, int step) {
            const bool on = step < last;
            const int k = 32 * step + 8 * fq;
#pragma unroll
            for (int f = 0; f < RF; ++f) {
                if constexpr (TRANS) {
                    const int p = 64 * f + lane, n = 32 * step + p / (2 * RF), r = r0 + 8 * (p % (2 * RF));
                    st.w[f] = __builtin_amdgcn_raw_buffer_load_b128(
                        wr, on && n < len && r < a.rank ? 2 * (n * a.rank + r) : -16, 0, 0);
                } else {
                    const int r = r0 + 16 * f + fi;
                    st.w[f] = __builtin_amdgcn_raw_buffer_load_b128(
                        wr, on && k < len && r < a.rank ? 2 * (r * len + k) : -16, 0, 0);
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int m = 16 * mt + fi;
                st.x[mt] = __builtin_amdgcn_raw_buffer_load_b128(
                    xr, on && k < len && m < rows ? 2 * (m * len + k) : -16, 0, 0);
            }
        };
        f32x4 acc[RF][MT];
#pragma unroll
        for (int f = 0; f < RF; ++f)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                acc[f][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        constexpr int kRing = 4;
        DnStep<RF, MT> ring[kRing];
#pragma unroll
        for (int i = 0; i < kRing; ++i)
            load(ring[i], first + wave + kDnWaves * i);
        for (int step = first + wave; step < last; step += kDnWaves * kRing) {
#pragma unroll
            for (int i = 0; i < kRing; ++i) {
                DnStep<RF, MT> &st = ring[i];
                u32x4 wf[RF];
                if constexpr (TRANS) {
                    // (one wave's LDS accesses run in order)
#pragma unroll
                    for (int f = 0; f < RF; ++f) {
                        const int p = 64 * f + lane;
                        *(u32x4 *)(stage + (p / (2 * RF)) * kPitch + 16 * (p % (2 * RF))) = st.w[f];
                    }
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int f = 0; f < RF; ++f) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int n = 8 * fq + 4 * u + (fi >> 2);
                            const v4i16 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                (__attribute__((address_space(3))) v4i16 *)(stage + n * kPitch + 32 * f +
                                                                            8 * (fi & 3)));
                            wf[f][2 * u] = (uint32_t)(uint16_t)q[0] | ((uint32_t)(uint16_t)q[1] << 16);
                            wf[f][2 * u + 1] = (uint32_t)(uint16_t)q[2] | ((uint32_t)(uint16_t)q[3] << 16);
                        }
                    }
                    __builtin_amdgcn_wave_barrier();
                } else {
#pragma unroll
                    for (int f = 0; f < RF; ++f)
                        wf[f] = st.w[f];
                }
#pragma unroll
                for (int f = 0; f < RF; ++f)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        acc[f][mt] = mfma<ACT>(wf[f], st.x[mt], acc[f][mt]);
                load(st, step + kDnWaves * (i + kRing));
            }
        }
        __syncthreads();  // (the last adapter's sums have been read)
#pragma unroll
        for (int f = 0; f < RF; ++f)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                red[wave][f][mt][lane] = acc[f][mt];
        __syncthreads();
        const float s = a.scale ? a.scale[ad] : 1.0f;
        for (int t = wave; t < RF * MT; t += kDnWaves) {
            const int f = t / MT, mt = t % MT;
            f32x4 v = red[0][f][mt][lane];
#pragma unroll
            for (int i = 1; i < kDnWaves; ++i) {
                const f32x4 u = red[i][f][mt][lane];
                v = f32x4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
            }
            const int r = r0 + 16 * f + 4 * fq;
            if (((mask[0] >> (16 * mt + fi)) & 1) && r < a.rank)
                *(f32x4 *)(part + ((int64_t)split * a.rows + m0 + 16 * mt + fi) * a.rank + r) =
                    f32x4{v[0] * s, v[1] * s, v[2] * s, v[3] * s};
        }
    }
}

// blockIdx: x the rows, y the part of the long axis, z slices of r, adapters'
// slots and (h, u) where both are wanted.
template <int ACT, int RF, int MT>
__global__ __launch_bounds__(kDnBlock) void down_kernel(DownArgs a)
{
    __shared__ f32x4 red[kDnWaves][RF][MT][64];
    __shared__ __attribute__((aligned(16))) char stages[kDnWaves * 32 * dn_pitch(RF)];
    int z = blockIdx.z;
    const int slice = z % a.slices;
    z /= a.slices;
    const int slot = z % a.slots;
    z /= a.slots;
    const bool trans = a.x ? z != 0 : true;
    if (trans)
        down<ACT, RF, MT, true>((const uint16_t *)a.dy, a, (const uint16_t *)a.b, a.u, a.N, slice, slot, blockIdx.y, red,
                                   stages);
    else
        down<ACT, RF, MT, false>((const uint16_t *)a.x, a, (const uint16_t *)a.a, a.h, a.K, slice, slot, blockIdx.y, red,
                                    stages);
}

template <int ACT, int RF>
hipError_t launch_dn(const DownArgs &a, const DownPlan &p, hipStream_t s)
{
    const dim3 grid((unsigned)p.tiles, (unsigned)a.parts,
                    (unsigned)(a.slices * a.slots * ((a.x ? 1 : 0) + (a.dy ? 1 : 0))));
    if (p.mt == 1)
        hipLaunchKernelGGL((down_kernel<ACT, RF, 1>), grid, dim3(kDnBlock), 0, s, a);
    else
        hipLaunchKernelGGL((down_kernel<ACT, RF, 2>), grid, dim3(kDnBlock), 0, s, a);
    return hipGetLastError();
}

template <int ACT>
hipError_t launch_dn_act(const DownArgs &a, const DownPlan &p, hipStream_t s)
{
    if (p.rf == 1)
        return launch_dn<ACT, 1>(a, p, s);
    if (p.rf == 2)
        return launch_dn<ACT, 2>(a, p, s);
    return launch_dn<ACT, 4>(a, p, s);
}

}  // namespace

DownPlan down_plan(int64_t rows, int64_t longest, int adapters, int rank, int both)
{
    DownPlan p;
    p.rf = rank <= 16 ? 1 : (rank <= 32 ? 2 : 4);
    p.slices = (rank + 16 * p.rf - 1) / (16 * p.rf);
    p.mt = rows <= 16 ? 1 : 2;
    p.tiles = (rows + 16 * p.mt - 1) / (16 * p.mt);
    // few rows: their adapters side by side
    const int64_t most = adapters < rows ? adapters : rows;
    p.slots = rows <= 64 ? (int)(most < 16 * p.mt ? most : 16 * p.mt) : 1;
    // parts: as many as give every compute unit two workgroups, at least 16
    // steps of 32 each, and no more than the kernels that add them up can take
    // in passing
    const int64_t blocks = p.tiles * p.slices * p.slots * (both ? 2 : 1);
    int64_t parts = 512 / (blocks ? blocks : 1), steps = (longest + 31) / 32;
    parts = parts < steps / 16 ? parts : steps / 16;
    p.parts = (int)(parts < 1 ? 1 : (parts > 8 ? 8 : parts));
    return p;
}

hipError_t launch_down(q4_dtype act_t, DownArgs a, const DownPlan &p, hipStream_t s)
{
    a.slices = p.slices;
    a.slots = p.slots;
    a.parts = p.parts;
    return act_t == Q4_BF16 ? launch_dn_act<Q4_BF16>(a, p, s) : launch_dn_act<Q4_F16>(a, p, s);
}

}  // namespace q4
