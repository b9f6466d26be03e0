/*
 * q4.h -- C ABI of libq4: 4-bit group-wise LLM weight quantization on AMD
 * Instinct MI355X (gfx950).
 *
 * Four operations: quantize fp16 weights to packed 4-bit codes plus per-group
 * metadata, dequantize them back to fp16/bf16, and multiply activations by
 * the quantized weights without materialising them (y = x . W^T), as a decode
 * GEMV (1 <= M <= 16) and a prefill GEMM (any M).  Beside them, the key/value
 * cache of a decoder in the same 4 bits: append, read back, attention over it
 * and eviction from it (q4_kv_*).
 *
 * Definitions this library implements (web pages on 4-bit group-wise
 * quantization, cited by title and section):
 *   - "What is 4-bit quantization and why does it matter?", "How 4-bit
 *     quantization works": quantized = round((w - zero_point) / scale),
 *     dequantized = quantized * scale + zero_point; INT4-symmetric levels
 *     -8..7 with an implicit zero and scale = max|w| / 7; NF4's 16 values
 *     (the printed table, used verbatim); weights stored as packed uint8 with
 *     the low nibble holding the earlier element; dequantize = table value
 *     times the block scale.
 *   - "INT4" (AI technologies atlas), "How it works" and "Components":
 *     asymmetric levels 0..15 with an integer zero-point; per-group scale
 *     usually stored in FP16; groups of 32, 64 or 128 weights.
 *   - "Loading a model in 4-bit", "Block-wise quantisation, stated exactly":
 *     contiguous blocks, absmax c = max|w| stored per block, each weight coded
 *     as the nearest of the 16 codebook entries after dividing by c,
 *     dequantized as c * Q[i]; "Where the accuracy goes": the layer
 *     dequantizes to the 16-bit compute dtype and runs an ordinary 16-bit
 *     matmul (fp32 accumulation here).
 *   - Double quantization of the NF4 absmax (Q4_NF4_DQ): the same page's
 *     double-quantization flag and "Where the accuracy goes" (the block
 *     constants are compressed as well), and its closing section on NF4 (the
 *     per-block scales quantized again in blocks of 256 to 8 bits, from 0.5
 *     to about 0.127 bits per parameter).  The 8-bit coding is not spelled
 *     out; it is read here as symmetric absmax int8 with a binary32 constant
 *     per run of 256 absmax values (rules below).
 *   - FP4 (Q4_FP4): "Loading a model in 4-bit", "Developer", names the fp4
 *     quant type beside nf4 without printing its codebook.  Read here as the
 *     E2M1 element values (bit 3 the sign, bits 2..1 an exponent e, bit 0 a
 *     mantissa bit m: m/2 for e = 0, else 2^(e-1) (1 + m/2), i.e. 0, 0.5, 1,
 *     1.5, 2, 3, 4, 6) divided by 6, each the nearest binary32, used exactly
 *     as NF4's table (block absmax, nearest entry).  Its agreement with any
 *     other fp4 implementation is not established by the pages.
 *
 * Data layout (all row-major, W is [N, K] like a Linear layer's weight):
 *   w       fp16 [N, K]
 *   codes   uint8 [N, K/2]; byte t of the flat array holds element 2t in its
 *           low nibble and element 2t+1 in its high nibble.
 *   scales  NF4, FP4: float32 [N, K/g] (the block absmax c)
 *           INT4-sym / INT4-asym: fp16 [N, K/g]
 *           NF4_DQ: bytes.  uint8 qc[N*K/g] (the 8-bit absmax codes in flat
 *           group order r*(K/g) + j), zero bytes up to the next multiple of
 *           16, then float32 s2[ceil(N*K/g / 256)] (one per run of 256
 *           groups in flat order; runs cross row boundaries).
 *   zeros   INT4-asym only: uint8 [ceil(N*K/g / 2)], the integer zero-points
 *           (0..15) of the groups in flat order r*(K/g) + j, two per byte,
 *           low nibble first.  NULL for the other formats.
 *   x       [M, K] fp16 or bf16 (act_t); y [M, N] in the same dtype.
 * A group is g contiguous elements of one row (K % g == 0).
 *
 * Coding rules (bit-exact, no fast-math; binary32 IEEE division by the
 * stored scale, round-half-even):
 *   NF4   c = max|w|; code = index of the nearest table entry to w / c, ties
 *         to the lower index; c == 0 gives code 7 (the entry 0.0).
 *   SYM   s = fp16(max|w| / 7); nibble = clamp(rint(w / s), -8, 7) + 8;
 *         s == 0 gives nibble 8.
 *   ASYM  lo = min(0, min w), hi = max(0, max w); s = fp16((hi - lo) / 15);
 *         z = clamp(rint(-lo / s), 0, 15); nibble = clamp(rint(w / s) + z,
 *         0, 15); s == 0 gives z = 0 and nibble 0.
 *   FP4   as NF4 with the FP4 table; ties to the lower index, so 0 codes as
 *         +0 (code 0); c == 0 gives code 0.
 *   NF4_DQ codes exactly as NF4 (with the exact absmax c); then per run of
 *         256 absmax values, s2 = c2 / 127 with c2 the run's max, and
 *         qc = clamp(rint(c / s2), 0, 127) (0 where s2 == 0).
 * Dequantize: NF4 and FP4 Q[i] * c, SYM (nibble - 8) * s, ASYM (nibble - z) * s, one
 * binary32 product rounded once (nearest-even) to fp16 or bf16.  NF4_DQ first
 * recovers c' = qc * s2 (one binary32 product), then Q[i] * c' as NF4.
 *
 * Conventions:
 *   - Ownership: every buffer is device memory owned by the caller.  The
 *     library never allocates, frees or retains memory, keeps no state
 *     between calls and never synchronises; it only enqueues kernels on
 *     `stream` (a hipStream_t; NULL selects the null stream).  Its globals
 *     are read-only constant tables, plus the per-GPU sync words of
 *     q4_gemv_chain_static (a static device array, and a host table of their
 *     addresses filled once per device under a lock); every other call is
 *     thread-safe, and overlapping q4_gemv_chain_static calls on one GPU
 *     race (see there).
 *   - Errors: every call validates its arguments on the host, before any HIP
 *     call, and returns a q4_status.  Nothing aborts and no C++ exception
 *     crosses the ABI.  Faults inside a kernel surface at the caller's next
 *     synchronisation.
 *   - Alignment: w, codes, x and out must be 16-byte aligned (the kernels
 *     move 16 bytes per lane); scales must be 4-byte (NF4, FP4), 2-byte (INT4) or
 *     16-byte (NF4_DQ) aligned, y 2-byte aligned.  There is no slow fallback path.
 *   - Preconditions not checked: inputs are finite; output buffers do not
 *     alias inputs; the buffers are at least the sizes q4_*_bytes report.
 */
#ifndef Q4_H
#define Q4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { Q4_NF4 = 0, Q4_INT4_SYM = 1, Q4_INT4_ASYM = 2, Q4_NF4_DQ = 3, Q4_FP4 = 4 } q4_format;
typedef enum { Q4_F16 = 0, Q4_BF16 = 1 } q4_dtype;
typedef enum {
    Q4_OK = 0,
    Q4_EINVAL = 1,       /* null pointer, N/K/M <= 0, K % g != 0, zeros given
                            (or missing) for the format */
    Q4_EUNSUPPORTED = 2, /* unknown format or dtype, g not in {32, 64, 128},
                            M > 16 for q4_gemv, a size beyond an entry
                            point's stated limit */
    Q4_EALIGN = 3,       /* a pointer violates the alignment rules above */
    Q4_EHIP = 4          /* the HIP runtime refused a launch */
} q4_status;

/* Sizes in bytes of the caller-allocated buffers for an [N, K] weight with
 * groups of g (0 for invalid arguments).
 *   codes:  exactly N*K/2.
 *   scales: the meaningful size -- N*(K/g)*4 (NF4, FP4), N*(K/g)*2 (INT4), or
 *           for NF4_DQ the 8-bit codes padded to a multiple of 16 plus
 *           4*ceil(N*(K/g)/256) -- plus P bytes of trailing padding;
 *   zeros:  the meaningful size ceil(N*(K/g)/2) (INT4-asym; 0 otherwise)
 *           plus P bytes of trailing padding;
 * where P = 16 + (the meaningful size rounded up to a multiple of 16, minus
 * the meaningful size), i.e. the total is the meaningful size plus 16,
 * rounded up to a multiple of 16.  Every entry point reads the meaningful
 * bytes only as values; q4_gemm with M > 16 fetches a row's scales and
 * zero-points for 256 columns at a time with wide loads that may start at
 * the last meaningful bytes and run into the padding, so a caller must
 * allocate the padded size (the padding's contents are never used and may
 * be anything).  q4_quantize writes only the meaningful bytes. */
size_t q4_codes_bytes(int64_t N, int64_t K);                      /* N*K/2 */
size_t q4_scales_bytes(q4_format f, int64_t N, int64_t K, int g); /* N*K/g * (4 NF4/FP4, 2 INT4), padded;
                                                                      NF4_DQ: qc, s2 as above, padded */
size_t q4_zeros_bytes(q4_format f, int64_t N, int64_t K, int g);  /* asym: ceil(N*K/g / 2), padded; else 0 */

/* Quantize fp16 weights w[N, K] into codes, scales and (asym) zeros.
 * Sources: the coding rules above ("How 4-bit quantization works";
 * "How it works" / "Components"; "Block-wise quantisation, stated exactly"). */
q4_status q4_quantize(q4_format f, int g, const void *w_f16, int64_t N, int64_t K,
                      uint8_t *codes, void *scales, uint8_t *zeros, void *stream);

/* Dequantize into out[N, K] of dtype out_t (fp16 or bf16).
 * Source: the dequantize rule above ("How 4-bit quantization works":
 * table value times the block scale; the affine inverse). */
q4_status q4_dequantize(q4_format f, int g, const uint8_t *codes, const void *scales,
                        const uint8_t *zeros, int64_t N, int64_t K, q4_dtype out_t,
                        void *out, void *stream);

/* Decode-shape product y[M, N] = x[M, K] . What^T for 1 <= M <= 16, reading
 * the packed weights once and dequantizing them in registers; fp32
 * accumulation, one rounding of y to act_t.  Every weight enters as the
 * value q4_dequantize writes in act_t, so the result equals a 16-bit matmul
 * on the dequantized weights up to summation order ("Where the accuracy
 * goes").  M = 1, 2 dequantize and multiply on the vector ALUs (binary32
 * dot products of 16-bit pairs) with one row per wave; 3 <= M <= 16 run as
 * a skinny product over blocks of 16 rows on the matrix cores.  M > 16
 * returns Q4_EUNSUPPORTED (use q4_gemm); K > Q4_GEMV_MAX_K returns
 * Q4_EUNSUPPORTED. */
#define Q4_GEMV_MAX_K 33554432
q4_status q4_gemv(q4_format f, int g, q4_dtype act_t, const void *x, int64_t M,
                  const uint8_t *codes, const void *scales, const uint8_t *zeros,
                  int64_t N, int64_t K, void *y, void *stream);

/* Prefill-shape product y[M, N] = x[M, K] . What^T for any M >= 1: weight
 * tiles are dequantized to the activation dtype on the fly (each value as
 * q4_dequantize writes it) and multiplied on the matrix cores with fp32
 * accumulation; y is rounded once to act_t ("Where the accuracy goes").
 * M <= 96 runs as the skinny product q4_gemv uses for 3 <= M <= 16, with
 * one, two or four blocks of 16 activation rows per launch (up to 64 rows)
 * and, past 64 rows, consecutive launches over row slices of x and y, all on
 * the caller's stream; 97 <= M <= 512 runs in tiles of 256 activation rows
 * by 128 weight rows, larger M in 256 x 256 tiles (the same bits either way).
 * K > Q4_GEMM_MAX_K returns Q4_EUNSUPPORTED. */
#define Q4_GEMM_MAX_K 4194304
q4_status q4_gemm(q4_format f, int g, q4_dtype act_t, const void *x, int64_t M,
                  const uint8_t *codes, const void *scales, const uint8_t *zeros,
                  int64_t N, int64_t K, void *y, void *stream);

/* Backward product through the frozen 4-bit weight, dX[M, K] = dY[M, N] .
 * What[N, K]: the gradient with respect to the layer input when the base
 * weights are quantized and frozen and only adapters train ("What is 4-bit
 * quantization and why does it matter?", "QLoRA fine-tunes in 4-bit": the
 * gradient flows through the dequantized weights, which never change).  Each
 * weight value is the one q4_dequantize writes in act_t; the products run on
 * the matrix cores with fp32 accumulation and dX is rounded once to act_t.
 * dy is [M, N], dx is [M, K], both act_t, row-major, 16-byte aligned.
 * Requires N % 8 == 0 (16-byte aligned dY rows), N <= Q4_GEMM_DX_MAX_N and
 * codes N*K/2 <= Q4_GEMV_CHAIN_MAX_CODES bytes, else Q4_EUNSUPPORTED. */
#define Q4_GEMM_DX_MAX_N 4194303
q4_status q4_gemm_dx(q4_format f, int g, q4_dtype act_t, const void *dy, int64_t M,
                     const uint8_t *codes, const void *scales, const uint8_t *zeros,
                     int64_t N, int64_t K, void *dx, void *stream);

/* A chain of decode GEMVs in one launch.  Each task is one M = 1 product
 * y[1, N] = x[1, K] . What^T with the layout and alignment rules of q4_gemv;
 * all tasks share the format, group size and activation dtype.  The tasks run
 * in order with the semantics of consecutive q4_gemv calls on the stream (and
 * the same bits in y): unless its flags hold Q4_TASK_NO_WAIT, a task reads x
 * only after every earlier task of the chain has written its y, so x may be
 * an earlier task's output.  Weights are read ahead across task boundaries,
 * so no task may write another task's weights.  Used for the weight stream of
 * a decode step, whose GEMVs are otherwise dominated by per-launch cost when
 * launched one by one ("Why it matters for deployment": a decode step reads
 * every weight once).
 *
 * ntasks is 1..Q4_GEMV_CHAIN_MAX; each K must satisfy K <= Q4_GEMV_CHAIN_MAX_K
 * and each task's codes N*K/2 <= Q4_GEMV_CHAIN_MAX_CODES bytes (else
 * Q4_EUNSUPPORTED); N and K are checked as in q4_gemv.  `sync` is a
 * device buffer of Q4_GEMV_CHAIN_SYNC_BYTES, 128-byte aligned, zeroed by the
 * caller before its first use: the kernel returns every word but word 2 to
 * zero when it ends, so the buffer can be reused without clearing by later
 * chains on the same stream; chains that may overlap (other streams) need
 * their own.  Word 2 becomes nonzero if a wait between tasks gave up after
 * about a second (the grid could not make progress; y is then undefined) and
 * stays set until the caller clears it.  The chain is one launch of one workgroup per
 * compute unit, cooperative when a task waits (its grid barrier needs every
 * workgroup resident): a launch the runtime refuses returns Q4_EHIP. */
#define Q4_GEMV_CHAIN_MAX 64
#define Q4_GEMV_CHAIN_MAX_K 16384
#define Q4_GEMV_CHAIN_MAX_CODES 2147483519LL /* 2^31 - 129 */
#define Q4_GEMV_CHAIN_SYNC_BYTES 1280 /* 10 lines of 128 bytes */
#define Q4_TASK_NO_WAIT 1u /* x is not written by earlier tasks: no grid-wide wait */
typedef struct {
    const void *x;        /* [1, K] act_t */
    const uint8_t *codes; /* [N, K/2] */
    const void *scales;   /* [N, K/g] */
    const uint8_t *zeros; /* asym: packed zero-points; else NULL */
    void *y;              /* [1, N] act_t */
    int64_t N, K;
    uint32_t flags;       /* 0 or Q4_TASK_NO_WAIT */
} q4_gemv_task;
q4_status q4_gemv_chain(q4_format f, int g, q4_dtype act_t, const q4_gemv_task *tasks,
                        int ntasks, uint32_t *sync, void *stream);

/* q4_gemv_chain without the sync buffer, for callers that cannot allocate
 * device memory (code under HIP graph capture, serving loops that forbid
 * allocation): the sync words live in a static device array of
 * Q4_GEMV_CHAIN_SYNC_BYTES that the library holds on each GPU it runs on
 * until the process ends.  Same tasks, limits, status codes and results as
 * q4_gemv_chain (the chain's size limits bound everything the array holds,
 * so no larger input needs more of it).  It calls no allocating routine:
 * the array's device address is looked up once per device, on the first
 * call with that device current, and a failed lookup returns Q4_EHIP.  The
 * kernel leaves the barrier counters at zero for the next call; the timeout
 * flag (word 2 of the sync words) is not reported.  All calls on one GPU
 * share the array: chains that may overlap on one GPU (different streams,
 * or one call still running while another is enqueued elsewhere) race and
 * must use q4_gemv_chain with their own sync buffers instead. */
q4_status q4_gemv_chain_static(q4_format f, int g, q4_dtype act_t, const q4_gemv_task *tasks,
                               int ntasks, void *stream);

/* ------------------------------------------------- the 4-bit key/value cache
 * Attention layers keep the keys and values of earlier tokens; here they are
 * held in the same 4 bits per value as the weights, and read by attention
 * without being written out.  The cache is a pool of pages: a page holds
 * `page` consecutive tokens of one sequence for every key/value head, and a
 * table gives each sequence's pages in order, so sequences grow and leave
 * without moving the others.
 *
 * Layout (row-major; `dim` values per row, a row being one token's key or
 * value in one head):
 *   k_codes, v_codes   uint8 [pages, heads, page, dim/2], low nibble first
 *   k_scales, v_scales [pages, heads, page, dim/g]: float32 (NF4, FP4) or
 *                      fp16 (INT4), as q4_quantize stores them for [N, dim]
 *   k_zeros, v_zeros   INT4-asym: uint8 [pages, heads, page, ceil(dim/g / 2)],
 *                      a row's zero-points two per byte, low nibble first (a
 *                      row starts a byte); NULL for the other formats
 * A group is g consecutive values of a row.  Coding and decoding follow the
 * rules above with w a row of fp16 or bf16 values, except that an INT4 scale
 * saturates at 65504 (bf16 rows can exceed fp16's range).  NF4_DQ is not
 * offered: its second-level constants span 256 groups, which arrive at
 * different times.
 *
 * Limits: dim 64, 128 or 256, g | dim; page 16, 32, 64, 128 or 256; up to
 * Q4_KV_MAX_LEN tokens a sequence.  Alignment: codes 16 bytes, scales 16,
 * zeros 4.  Memory past a sequence's length (the rest of its last page) and
 * pages no table names may hold anything, NaN scales included. */
#define Q4_KV_MAX_LEN 4194304
typedef struct {
    uint8_t *k_codes;
    void *k_scales;
    uint8_t *k_zeros;
    uint8_t *v_codes;
    void *v_scales;
    uint8_t *v_zeros;
    int64_t pages; /* in the pool */
    int32_t page;  /* tokens per page */
    int32_t heads; /* key/value heads */
    int32_t dim;   /* values per row */
    int32_t g;     /* group size */
    int32_t format; /* q4_format */
    int32_t reserved; /* 0 */
} q4_kv_cache;

/* A batch: `seqs` sequences, each with some new tokens at its end.  The new
 * tokens' rows are packed: those of sequence b are rows starts[b] ..
 * starts[b+1] - 1 of the packed arrays, its i-th new token at position
 * lens[b] - (starts[b+1] - starts[b]) + i (starts NULL: one token each, row b).
 * lens counts the new tokens.  Table, lens and starts are device arrays, read
 * by the kernels; max_new and max_len are upper bounds the caller knows
 * (they shape the launches; a sequence is taken to end at max_len if lens
 * says more).  A new token whose position is negative sees no key (and is not
 * stored); a table entry outside 0 .. pages - 1 is never followed: its tokens
 * are not stored, read as zero, and take no part in attention. */
typedef struct {
    const int32_t *table;  /* [seqs, table_width] page numbers */
    const int32_t *lens;   /* [seqs] */
    const int32_t *starts; /* [seqs + 1], or NULL */
    int64_t tokens;        /* rows of the packed arrays */
    int32_t table_width;
    int32_t seqs;
    int32_t max_new;       /* most new tokens of a sequence */
    int32_t max_len;       /* at least every lens[b]; <= table_width * page */
} q4_kv_batch;

/* Code the new tokens' keys and values into their pages.  k and v are
 * [tokens, heads, dim] of in_t with the given distances between tokens and
 * between heads in elements (multiples of 8; a row itself is contiguous). */
q4_status q4_kv_append(const q4_kv_cache *cache, const q4_kv_batch *batch, q4_dtype in_t,
                       const void *k, int64_t k_token_stride, int64_t k_head_stride,
                       const void *v, int64_t v_token_stride, int64_t v_head_stride, void *stream);

/* The new tokens' keys and values as they stand in the cache, dequantized to
 * contiguous [tokens, heads, dim] arrays of out_t: one binary32 product
 * rounded once, as q4_dequantize. */
q4_status q4_kv_read(const q4_kv_cache *cache, const q4_kv_batch *batch, q4_dtype out_t, void *k,
                     void *v, void *stream);

/* Attention of the new tokens over their sequences' cached tokens.
 *   q    [tokens, q_heads, dim] of act_t, strides as in q4_kv_append;
 *        q_heads = G heads with 1 <= G <= Q4_KV_MAX_GROUP, query head j
 *        reading key/value head j / G
 *   out  [tokens, q_heads, dim] of act_t, contiguous, 16-byte aligned
 *   lse  float32 [tokens, q_heads] or NULL: log of the softmax denominator
 *   mass float32 [seqs, heads, mass_width] or NULL, mass_width >= max_len:
 *        mass[b, h, t] += the softmax weights that the rows of head h's
 *        query heads put on token t, all new tokens together
 * A token at position p sees the tokens t with t <= p and, for window > 0,
 * t > p - window.  With x_t = scale * <q, K_t>: out = sum_t softmax(x)_t V_t.
 * A row that sees nothing gives out = 0 and lse = -infinity.  0 < scale <= 2^60.
 * Scores, softmax statistics, sums and masses are binary32; the result does not
 * depend on timing (no floating-point atomics).  In the product with the values
 * the weights are fp16 (act_t fp16: in two parts, of 22 bits together), and
 * where a head has many rows (more than 32 times g / dim, dim 64: 64 times) so
 * are the values, relative to their token's largest scale: groups down to
 * 2^-21 of it keep 11 bits, and so do weights that, times their token's scale,
 * are 2^-23 of the row's largest.  What a row does not see changes nothing of
 * that.  (An fp16 output is 2.1e-4 to 2.8e-4 off in relative 2-norm, where
 * rounding it alone leaves 2.1e-4; a bf16 output 1.7e-3, its rounding.)  Of what
 * a cache holds it is assumed that scales are not negative and |value| < 2^60.
 * workspace: device memory of q4_kv_workspace_bytes (for the same window and
 * with_mass = (mass != NULL)), 256-byte aligned, needed
 * until the call's work has run; its contents before and after do not matter
 * (calls that may overlap need their own). */
#define Q4_KV_MAX_GROUP 64
size_t q4_kv_workspace_bytes(const q4_kv_cache *cache, const q4_kv_batch *batch, int q_heads,
                             int window, int with_mass);
q4_status q4_kv_attention(const q4_kv_cache *cache, const q4_kv_batch *batch, q4_dtype act_t,
                          const void *q, int64_t q_token_stride, int64_t q_head_stride,
                          int q_heads, float scale, int window, void *out, float *lse,
                          float *mass, int64_t mass_width, void *workspace,
                          size_t workspace_bytes, void *stream);

/* Eviction by accumulated attention weight.  Per sequence and head, the tokens
 * that stay are: all of them if they are at most `budget`; otherwise the last
 * `recent` tokens and the budget - recent others of largest mass (equal
 * masses: the earlier token; NaN counts below every number).  Tokens whose
 * page number is outside the pool are not there: they never stay, and none of
 * these counts takes them in.  The tokens that stay move, in
 * token order, to slots 0, 1, ... of the pages new_table names, with their
 * mass; codes, scales and zero-points are copied as they are.
 * batch: table, lens, seqs and max_len are used; starts, tokens and max_new
 * are not.  new_table [seqs, new_table_width] names pages of the same pool,
 * none of them in use by the sequences that are read.  0 <= recent <= budget.
 *   new_lens int32 [seqs]: the number of tokens that stay (in every head the
 *            same): min(lens[b], budget), where all pages exist
 *   new_mass float32 [seqs, heads, new_width], new_width >= budget: the kept
 *            tokens' masses, then zeros; not overlapping mass
 *   kept     int32 [seqs, heads, budget]: the kept tokens' positions, then -1 */
q4_status q4_kv_evict(const q4_kv_cache *cache, const q4_kv_batch *batch, const float *mass,
                      int64_t mass_width, const int32_t *new_table, int new_table_width,
                      int budget, int recent, int32_t *new_lens, float *new_mass,
                      int64_t new_width, int32_t *kept, void *stream);

/* A static, human-readable name for a status code. */
const char *q4_status_str(q4_status s);

#ifdef __cplusplus
}
#endif

#endif /* Q4_H */
