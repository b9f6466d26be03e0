// q4_internal.hpp -- launchers shared between the C-ABI front end
// (q4_api.hip) and the kernel files.  Arguments arrive validated.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "plan.hpp"
#include "q4.h"

namespace q4 {

// Number of compute units of the current device (queried per call).
int device_cu_count();

// Allocated size of a scale or zero-point array of n meaningful bytes: at
// least 16 bytes of padding, to a multiple of 16, so that loads of up to 16
// bytes starting at any meaningful byte stay inside the allocation.
__host__ __device__ constexpr int64_t padded_meta_bytes(int64_t n)
{
    return (n + 16 + 15) & ~(int64_t)15;
}

// NF4_DQ scales buffer: byte offset of the float32 second-level constants
// (one per kDqRun groups, flat order) after the n_groups 8-bit codes.
constexpr int kDqRun = 256;
__host__ __device__ constexpr int64_t dq_s2_offset(int64_t n_groups)
{
    return (n_groups + 15) & ~(int64_t)15;
}
__host__ __device__ constexpr int64_t dq_scales_bytes(int64_t n_groups)
{
    return dq_s2_offset(n_groups) + 4 * ((n_groups + kDqRun - 1) / kDqRun);
}

hipError_t launch_quantize(q4_format f, int g, const void *w, int64_t N, int64_t K,
                           uint8_t *codes, void *scales, uint8_t *zeros, hipStream_t s);
hipError_t launch_dequantize(q4_format f, int g, const uint8_t *codes, const void *scales,
                             const uint8_t *zeros, int64_t N, int64_t K, q4_dtype out_t,
                             void *out, hipStream_t s);
hipError_t launch_gemv(q4_format f, int g, q4_dtype act_t, const void *x, int64_t M,
                       const uint8_t *codes, const void *scales, const uint8_t *zeros,
                       int64_t N, int64_t K, void *y, hipStream_t s);
// Skinny product on the matrix cores: up to 64 activation rows per launch,
// more as consecutive launches over row slices.
hipError_t launch_gemv_mfma(q4_format f, int g, q4_dtype act_t, const void *x, int64_t M,
                            const uint8_t *codes, const void *scales, const uint8_t *zeros,
                            int64_t N, int64_t K, void *y, hipStream_t s);
// Chained M = 1 GEMVs (at most Q4_GEMV_CHAIN_MAX tasks per launch).
bool gemv_chain_k_ok(int64_t K);
hipError_t launch_gemv_chain(q4_format f, int g, q4_dtype act_t, const q4_gemv_task *tasks,
                             int ntasks, uint32_t *sync, hipStream_t s);
// Backward product dX = dY . What (QLoRA's gradient through the frozen weights).
hipError_t launch_gemm_dx(q4_format f, int g, q4_dtype act_t, const void *dy, int64_t M,
                          const uint8_t *codes, const void *scales, const uint8_t *zeros,
                          int64_t N, int64_t K, void *dx, hipStream_t s);
hipError_t launch_gemm(q4_format f, int g, q4_dtype act_t, const void *x, int64_t M,
                       const uint8_t *codes, const void *scales, const uint8_t *zeros,
                       int64_t N, int64_t K, void *y, hipStream_t s);
// The same with 128-row weight tiles (4 waves per workgroup), for middle M.
hipError_t launch_gemm_bn128(q4_format f, int g, q4_dtype act_t, const void *x, int64_t M,
                       const uint8_t *codes, const void *scales, const uint8_t *zeros,
                       int64_t N, int64_t K, void *y, hipStream_t s);

// A product through experts' weights, one array of experts * N rows: row r of
// group e (rows offsets[e] .. offsets[e + 1] - 1 of `rows`) is x's row index[r]
// (r without an index), of xrows, against the N rows of expert e.
struct ExpertsArgs {
    const void *x;
    int64_t xrows;
    const int32_t *index, *offsets;
    int64_t rows;
    int experts;
    const uint8_t *codes;
    const void *scales;
    const uint8_t *zeros;
    int64_t N, K;
    void *y;
};
hipError_t launch_experts(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s);
// Pieces of up to 16 rows of an expert a workgroup.
hipError_t launch_experts_skinny(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s);
// Pieces of up to 16 mt (1 or 2) rows by resident workgroups, for K up to
// kStreamMaxK and up to kStreamMaxCodes bytes of codes an expert.
hipError_t launch_experts_stream(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, int mt, hipStream_t s);
// Tiles of up to 64, 128 or 256 rows of an expert.
hipError_t launch_experts_tile64(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s);
hipError_t launch_experts_tile128(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s);
hipError_t launch_experts_tile256(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s);
// The gradient dX[r] = dY[r] . What_e: x is dY, y is dX.
hipError_t launch_experts_dx(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s);

// Low-rank adapters beside a weight: h[m] = scale x[m] A^T and u[m] = scale
// dy[m] B of each row's adapter (x or dy NULL: h or u is not formed), as the
// plan says in binary32 partial sums [parts, rows, rank] or as three bfloat16
// parts [rows, 3, rank] (LowRank in lora.hpp).
struct DownArgs {
    const void *x, *dy, *a, *b;
    const float *scale;
    const int32_t *ids;
    void *h, *u;
    float *sums;  // [h, u][parts, rows, rank]: of the parts where they are joined
    int64_t rows;
    int N, K, adapters, rank;
    int slices, slots, parts;  // of the plan
};
hipError_t launch_down(q4_dtype act_t, DownArgs a, const DownPlan &p, hipStream_t s);

// The products with the adapters' part added: y = x What^T + h B^T and dX = dY
// What + u A.
struct LoraArgs {
    const void *x;  // or dY
    int64_t M;
    const uint8_t *codes;
    const void *scales;
    const uint8_t *zeros;
    int64_t N, K;
    const void *w;  // B [adapters, N, rank], or A [adapters, rank, K]
    const int32_t *ids;
    int adapters, rank;
    const void *low;  // h or u as launch_down leaves it
    int parts;
    void *y;  // or dX
    // the contraction (dX; y in tiles of 64 rows) in so many parts, whose sums go
    // here, [out_parts, M, K] or [out_parts, M, N up to a multiple of 4]
    int out_parts;
    float *sums;
};
hipError_t launch_lora_skinny(q4_format f, int g, q4_dtype act_t, const LoraArgs &a, hipStream_t s);
hipError_t launch_lora_tile64(q4_format f, int g, q4_dtype act_t, const LoraArgs &a, hipStream_t s);
hipError_t launch_lora_tile128(q4_format f, int g, q4_dtype act_t, const LoraArgs &a, hipStream_t s);
hipError_t launch_lora_tile256(q4_format f, int g, q4_dtype act_t, const LoraArgs &a, hipStream_t s);
hipError_t launch_lora_dx(q4_format f, int g, q4_dtype act_t, const LoraArgs &a, hipStream_t s);

// The adapters' gradients, dA[a] = sum u[m]^T x[m] and dB[a] = sum dy[m]^T
// h[m] over the rows m of adapter a, in `splits` parts of the rows (more than
// one: sums in `sums`, which launch_lora_grad joins).
struct GradArgs {
    const void *x, *dy;
    const int32_t *ids;
    const uint16_t *h, *u;  // three parts each
    float *sums;
    int64_t rows;
    int N, K, adapters, rank, splits;
    void *da, *db;
};
hipError_t launch_lora_grad(q4_dtype act_t, const GradArgs &a, hipStream_t s);

}  // namespace q4
