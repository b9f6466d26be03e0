// plan.hpp -- how the products of rows in groups are cut up: the kernel that a
// call's sizes choose, its parts, and the workspace that those need.  Host
// arithmetic alone, without HIP, so that a program without a card can ask it.
#pragma once

#include <cstdint>

namespace q4 {

// ------------------------------------------------------------------ experts
// K, and bytes of codes an expert, up to which resident workgroups stream the
// products of few rows.
constexpr int64_t kStreamMaxK = 4096, kStreamMaxCodes = 0x7fff0000;

// Few rows: resident workgroups with pieces of up to 16 or 32 rows, or (skinny)
// a workgroup for each block of weight rows; more: tiles of up to so many rows.
enum class ExpertsKernel { stream1, stream2, skinny, tile64, tile128, tile256 };

// The kernel by the mean number of rows an expert has (of the experts that can
// have any).  Times in us, one card, bf16 rows, uneven groups; a: 64 experts of
// 2048 x 4096 INT4-asym g 32, b: 16 of 4096 x 4096 NF4 g 64, c: 64 of 1024 x 2048
// INT4-sym g 64, d: 8 of 4096 x 14336 NF4 g 64, e: 64 of 1024 x 4096 NF4 g 64, f: 8
// of 1024 x 4096 INT4-sym g 64:
//   mean               4     8    12    16    24    32    48    64    96   128
//   a one block       75    90   103   117   147   185   245
//     two blocks      77    93   100   106   123   137   171
//     64 rows        114   120   125   129   147   157   171   228   310   367
//     128 rows       115   121   124   127   130   151   152   175   196   258
//     256 rows                                           142   181   204   231
//   b one block       36    43    51    59    66    86   112
//     two blocks      42    46    59    61    68    76    96
//     64 rows         50    50    51    52    52    55    76    88   122   168
//     128 rows        50    50    51    51    52    53    80    83    91   107
//     256 rows                                            78    80    84   104
//   c one block       23    25    29    32    40    46    62
//     two blocks      24    25    30    32    37    40    48
//     64 rows         25    26    26    26    37    38    41    45    59    79
//     128 rows        25    26    26    27    28    41    42    45    48    52
//     256 rows                                            47    48    51    55
//   d skinny          81   112   125   166   207   269   373
//     64 rows        107   132   133   142   139   146   180   182   201   295
//     128 rows       107   138   138   141   139   145   209   171   201   218
//     256 rows                                           247   212   292   293
//   e one block       39    48    53    61    74    87   118
//     two blocks      47    56    62    64    75    82   102
//     64 rows         49    50    52    52    74    75    79    94   140   161
//     128 rows        49    51    51    52    79    59    82    89   109   136
//     256 rows                                            78    81   103   114
//   f two blocks      14    12    14    15    24    29    33
//     64 rows         30    30    30    30    32    33    33    33    33    33
//     128 rows        30    30    30    30    32    36    39    39    39    40
//   mean             192   256   (128 / 256 rows)
//   a            434/296   563/340
//   b            206/187   277/195
// The few rows' kernels win or tie up to 12 rows on all but c (29 against 26); from
// 16 on tiles do on b to e, two blocks on a up to 24 and on f, whose blocks are
// few, up to 32.
inline ExpertsKernel experts_kernel(int64_t rows, int64_t experts, int64_t N, int64_t K)
{
    const int64_t mean = rows / (experts < rows ? experts : rows);
    if (mean <= 12) {
        if (K <= kStreamMaxK && N * (K / 2) <= kStreamMaxCodes)
            return mean < 8 ? ExpertsKernel::stream1 : ExpertsKernel::stream2;
        return ExpertsKernel::skinny;
    }
    // 64-row tiles where those of 128, the rows counted as one group, would be
    // fewer than 128: with few experts they leave half of the compute units idle
    // (f; d at 48 rows; 2 of 298 x 6496 INT4-asym, 256 rows: 76 / 60 us).  Many
    // small groups make more tiles than that, but then both kernels run most of
    // their pieces as the same 64-row tiles: b and e within 7 %, c at 24 rows 37 / 28.
    const int64_t tiles = (rows + 127) / 128 * ((N + 127) / 128);
    if (tiles < 128)
        return ExpertsKernel::tile64;
    return mean < 160 || tiles < 512 ? ExpertsKernel::tile128 : ExpertsKernel::tile256;
}

// The gradient: pieces of 256 rows, or of 64 where those are too few to fill the
// card (1694 rows of 5 experts of 5864 x 256 INT4-sym g 32: 91 -> 55 us).
inline int experts_dx_rows(int64_t rows, int64_t K)
{
    return (rows + 255) / 256 * ((K + 127) / 128) <= 64 ? 64 : 256;
}

// ----------------------------------------------------------------- adapters
// Most parts that h is left in (the readers hold so many loads in flight).
constexpr int kMostParts = 8;

// How h and u are formed: a tile of rows, 16 rf values r and one of `parts`
// parts of the long axis a workgroup, the adapters of a tile over `slots`
// workgroups.  split: left as three 16-bit parts, the parts of the axis joined.
struct DownPlan {
    bool split;
    int rf, slices, slots, parts;
    int64_t tiles;
};
// A workgroup's rows and a step of the axis, where rows are not few.
constexpr int kDownRows = 64, kDownStep = 64;
inline DownPlan down_plan(int64_t rows, int64_t longest, int adapters, int rank, int backward)
{
    DownPlan p;
    p.split = backward || rows > 96;  // (96: as far as the skinny product goes)
    p.rf = rank <= 16 ? 1 : (rank <= 32 ? 2 : 4);
    p.slices = (rank + 16 * p.rf - 1) / (16 * p.rf);
    const int tile = p.split ? kDownRows : 16;
    p.tiles = (rows + tile - 1) / tile;
    // few rows: their adapters side by side.  Whole calls on 4096 x 4096 in us, a
    // tile's adapters one after another / on up to 16 workgroups; product, then
    // backward.  100 rows of 32 adapters of rank 16 in any order 95 / 40, 124 / 68;
    // of 4 34 / 28, 43 / 36; 512 rows of 32 in any order 121 / 66, 177 / 126, in runs
    // 51.5 / 45.4, 82 / 81.  Beyond 512 workgroups without rows of theirs cost runs
    // (1024 rows of 32 adapters 77.9 / 79.4, 90 / 99; 2048 104 / 112, 121 / 130) what
    // rows in any order would gain (1024 171 / 125, 218 / 184; 2048 205 / 169, 383 / 295).
    const int64_t most = adapters < rows ? adapters : rows;
    p.slots = rows <= 512 ? (int)(most < 16 ? most : 16) : 1;
    if (p.slots < 1)
        p.slots = 1;
    // parts of the long axis: as many as give every compute unit two
    // workgroups, of at least 16 (few rows) or 8 steps each; with up to 16
    // steps of 64 the join's launch would cost more than it saves
    const int64_t blocks = p.tiles * p.slices * p.slots * (backward ? 2 : 1);
    const int64_t steps = p.split ? (longest + kDownStep - 1) / kDownStep : (longest + 31) / 32;
    const int64_t most_parts = p.split ? (steps <= 16 ? 1 : steps / 8) : steps / 16;
    int64_t parts = 512 / (blocks ? blocks : 1);
    parts = parts < most_parts ? parts : most_parts;
    p.parts = (int)(parts < 1 ? 1 : (parts > kMostParts ? kMostParts : parts));
    return p;
}

// Whether a product of more than 96 rows runs in tiles of 64 (q4_lora_gemm).
inline bool short_tiles(int64_t M, int64_t N) { return M > 96 && (M + 255) / 256 * ((N + 127) / 128) < 128; }

// Parts of K for them: as many as give every compute unit a workgroup, of at
// least 8 steps of 64.  Whole calls in us, whole / in parts: 237 rows of 147 x
// 5888, rank 88, 60 / 26; 835 of 553 x 8064, rank 80, 85 / 45; 128 of 512 x 14336,
// rank 16, 117 / 33; 128 of 4096 x 4096 42 / 28; 697 of 394 x 1472, rank 112, 29 /
// 24; 512 of 4096 x 4096 46 / 44.
inline int lora_parts(int64_t M, int64_t N, int64_t K)
{
    const int64_t tiles = (M + 63) / 64 * ((N + 127) / 128);
    if (!short_tiles(M, N) || tiles >= 256)
        return 1;
    const int64_t parts = 256 / tiles, most = (K + 255) / 256 / 2;
    return (int)(parts < most ? parts : (most > 1 ? most : 1));
}

// The product's kernel by the number of rows, as q4_gemm's, but for tiles that
// would leave half of the compute units idle (835 rows of 553 x 8064, rank 80:
// 199 -> 80 us in tiles of 64 rows, without parts; 619 of 682 x 1920, rank 24: 83
// -> 35).
enum class LoraKernel { skinny, tile64, tile128, tile256 };
inline LoraKernel lora_kernel(int64_t M, int64_t N)
{
    if (M <= 96)
        return LoraKernel::skinny;
    if (short_tiles(M, N))
        return LoraKernel::tile64;
    return M <= 512 || (M + 255) / 256 * ((N + 255) / 256) < 128 ? LoraKernel::tile128 : LoraKernel::tile256;
}

// The gradient's tiles are of 128 columns, its steps of 64 weight rows.
constexpr int kDxCols = 128, kDxStep = 64;
// Tiles of 256 rows, or of 128 or 64 where those too are one round of
// workgroups or less (256 compute units): a short tile takes less time, but a
// weight's column is dequantized once a tile.  dX alone, rank 16, in us, with
// tiles of 256 / 128 / 64 rows: 512 rows of 4096 x 4096 NF4 g 64 (64 tiles of
// 256) 80 / 64 / 57, 768 rows (96) 81 / 64 / 100, 1024 rows (128) 81 / 65 / 100;
// 333 rows of 1024 x 1024 (16) 30 / 23 / 20.
inline int lora_dx_rows(int64_t M, int64_t K)
{
    const int64_t tiles = (M + 255) / 256 * ((K + kDxCols - 1) / kDxCols);
    return tiles <= 64 ? 64 : (tiles <= 128 ? 128 : 256);
}

// Parts of N: as many as give every compute unit a workgroup, of at least 8
// steps.  dX alone in us, NF4 g 64, rank 16, whole / in parts of at least 16 / of
// 8 steps: 1 row, N 7640, K 1024 89 / 27 / 24; 16 rows of 4096 x 4096 53 / 26 / 23; 64 of 14336 x 4096 162 / 43 / 42; 16 of 2048 x 4096 32 / 25 /
// 21; 333 of 4096 x 2048 55 / 39 / 39; 333 of 1024 x 1024 (16 steps) 19.6 / 19.6 / 18.8.
inline int lora_dx_parts(int64_t M, int64_t N, int64_t K)
{
    const int64_t tiles = (M + 63) / 64 * ((K + kDxCols - 1) / kDxCols), steps = (N + kDxStep - 1) / kDxStep;
    const int64_t parts = tiles > 0 && tiles < 256 ? 256 / tiles : 1, most = steps / 8;
    return (int)(parts < most ? parts : (most > 1 ? most : 1));
}

// The adapters' gradients: a workgroup takes 128 columns and up to 16 rf values
// r, 64 rows a step.
constexpr int kGrRows = 64, kGrCols = 128;
inline int grad_rf(int rank) { return rank <= 16 ? 1 : (rank <= 32 ? 2 : 4); }
// Parts of the rows: as many as give every compute unit two workgroups, at
// least four steps each, at most 8 (their sums are written and read).
inline int grad_splits(int64_t rows, int64_t N, int64_t K, int adapters, int rank)
{
    const int rf = grad_rf(rank), slices = (rank + 16 * rf - 1) / (16 * rf);
    const int64_t blocks = ((K + kGrCols - 1) / kGrCols + (N + kGrCols - 1) / kGrCols) * adapters * slices;
    const int64_t steps = (rows + kGrRows - 1) / kGrRows;
    int64_t n = 512 / blocks;
    n = n < steps / 4 ? n : steps / 4;
    return (int)(n < 1 ? 1 : (n > 8 ? 8 : n));
}

inline int64_t padded(int64_t floats) { return (4 * floats + 255) / 256 * 256; }

// The workspace: h, then (backward) u, then sums that are joined: of the parts
// of h and u, later of y or of dX and of the adapters' gradients.
struct LoraLayout {
    DownPlan plan;
    int splits, out_parts;
    int64_t u, sums, bytes;
};
inline LoraLayout lora_layout(int64_t M, int64_t N, int64_t K, int adapters, int rank, int backward)
{
    LoraLayout w{};
    w.plan = down_plan(M, backward && N > K ? N : K, adapters, rank, backward);
    // (three 16-bit parts are as long as one and a half of 32; rank is even)
    const int64_t one = padded(w.plan.split ? M * rank / 2 * 3 : w.plan.parts * M * rank);
    const int kinds = backward ? 2 : 1;
    w.splits = backward ? grad_splits(M, N, K, adapters, rank) : 1;
    w.u = one;
    w.sums = kinds * one;
    const int64_t joined = w.plan.split && w.plan.parts > 1 ? padded((int64_t)kinds * w.plan.parts * M * rank) : 0;
    const int64_t grads = w.splits > 1 ? padded((int64_t)w.splits * adapters * rank * (N + K)) : 0;
    w.out_parts = backward ? lora_dx_parts(M, N, K) : lora_parts(M, N, K);
    const int64_t out = w.out_parts > 1 ? padded(w.out_parts * M * (backward ? K : (N + 3) / 4 * 4)) : 0;
    const int64_t most = joined > grads ? joined : grads;
    w.bytes = w.sums + (most > out ? most : out);
    return w;
}

}  // namespace q4
