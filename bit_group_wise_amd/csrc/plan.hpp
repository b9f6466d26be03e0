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
// have any).  Times in us, one card; a: 64 experts of 2048 x 4096 INT4-asym g
// 32, b: 16 of 4096 x 4096 NF4 g 64, c: 64 of 1024 x 2048 INT4-sym g 64, d: 8
// of 4096 x 14336 NF4 g 64; bf16 rows, uneven groups:
//   mean                 4             8            12            16            24
//   one block   a 80  b 39   a 96  b 42   a 105  b 53   a 118  b 60   a 151  b 77
//   two blocks  a 83  b 46   a 89  b 53   a 103  b 55   a 109  b 64   a 121  b 77
//   128 rows                 a 123 b 53   a 126  b 56   a 128  b 58   a 147  b 67
//   two, 128    c 24         c 24  c 26   c 30   c 26   c 32   c 27   c 35   c 32
//   skinny, 128 d 112        d 108 d 141  d 128  d 148  d 157  d 148  d 206  d 156
//   mean                96           128           192           256
//   128 rows    a 207  b 101  a 250  b 124  a 434  b 206  a 563  b 277
//   256 rows    a 229  b 141  a 238  b 145  a 296  b 187  a 340  b 195
inline ExpertsKernel experts_kernel(int64_t rows, int64_t experts, int64_t N, int64_t K)
{
    const int64_t mean = rows / (experts < rows ? experts : rows);
    if (mean <= 12) {
        if (K <= kStreamMaxK && N * (K / 2) <= kStreamMaxCodes)
            return mean < 8 ? ExpertsKernel::stream1 : ExpertsKernel::stream2;
        return ExpertsKernel::skinny;
    }
    // tiles that would leave half of the compute units idle are cut: 2 experts of
    // 298 x 6496 INT4-asym, 333 rows: 164 -> 63 us
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
    // few rows: their adapters side by side
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
