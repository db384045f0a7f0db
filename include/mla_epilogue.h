/*
 * mla_epilogue.h -- C ABI of the fused MLA decode epilogue for NVIDIA B200 (sm_100a).
 *
 * The operation (vLLM PR #54896 report on prhub.com.cn, sections 实现拆解
 * "implementation" items 1-3 and 关键源码片段 "key source snippets":
 * fusedKimiK3MLADecodeQConcatKVCacheKernel / writeLatent576 and the
 * launcher fused_kimi_k3_mla_decode_q_concat_kv_cache_insert):
 *
 *   for every token t < T:
 *     for every head h < H:   q_out[t, h, :]            = enc_q (rope(q_nope[t, h, :] || q_pe[t, h, :]))
 *     if slot_mapping[t] ok:  cache.row(slot_mapping[t]) = enc_kv(rope(kv_c[t, :]    || k_pe[t, :]))
 *
 * where every row is 576 = 512 (latent "nope") + 64 (rotary "pe") wide;
 * rope() turns each pair (x[512+i], x[544+i]), i < 32, of the pe part by the
 * angle whose cosine and sine are cos_sin[positions[t]][i] and
 * cos_sin[positions[t]][32+i] (rotate-half RoPE, computed in fp32 as
 * (a c - b s, b c + a s), each product and the sum rounded separately) and
 * leaves the 512 nope values unchanged; enc is a round-to-nearest-even bf16
 * store, or, with the matching FP8 flag, the OCP E4M3FN byte
 * satfinite_rn(y / scale) of the fp32 value y (IEEE fp32 division, no
 * intermediate bf16 rounding).  Without RoPE and FP8 the call is a plain
 * concatenation plus cache scatter, bit for bit.
 *
 * Conventions for every entry point below:
 *   - all data pointers are DEVICE pointers; the caller allocates and owns
 *     every buffer; no entry point allocates, frees or synchronises;
 *   - work is enqueued on `stream` (0 = the legacy default stream) and runs
 *     asynchronously; a return of MLA_OK means "launched", not "finished";
 *   - strides are in ELEMENTS; the innermost stride of every row is 1;
 *   - host-side argument errors return a status and launch nothing.  Index
 *     values that live in device memory (slots, positions) are range-checked
 *     by the kernel, which skips what is out of range and reports it through
 *     the optional status word; it never faults or traps on them.
 */
#ifndef MLA_EPILOGUE_H
#define MLA_EPILOGUE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define MLA_API __attribute__((visibility("default")))
#else
#define MLA_API
#endif

/* Same type as cudaStream_t, declared here so that this header needs no CUDA include. */
typedef struct CUstream_st* mla_stream_t;

typedef enum mla_status {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1, /* null pointer, negative or too-large size, bad stride, conflicting flags */
  MLA_ERR_ALIGNMENT = 2,   /* a pointer or stride breaks the alignment rules below */
  MLA_ERR_UNSUPPORTED = 3, /* an unknown flag bit */
  MLA_ERR_CUDA = 4         /* the CUDA runtime refused the launch; see mla_last_cuda_error() */
} mla_status;

/* flags */
#define MLA_FLAG_ROPE        1u  /* rotate the 64 pe dims (needs positions, cos_sin) */
#define MLA_FLAG_Q_FP8       2u  /* q_out is e4m3 bytes, scaled by *q_scale (needs q_scale) */
#define MLA_FLAG_KV_FP8      4u  /* cache is e4m3 bytes, scaled by *kv_scale (needs kv_scale) */
#define MLA_FLAG_PDL         8u  /* launch as a programmatic dependent of the previous kernel on `stream` */
#define MLA_FLAG_FORCE_SPLIT 16u /* use MLA_MODE_SPLIT whatever T is (tests, tuning) */
#define MLA_FLAG_FORCE_ROWS  32u /* use MLA_MODE_ROWS whatever T is (tests, tuning); not with FORCE_SPLIT */

/* bits the kernel ORs into *status */
#define MLA_STATUS_SLOT_RANGE 1  /* some slot_mapping[t] >= num_blocks*block_size: that cache row was not written */
#define MLA_STATUS_POS_RANGE  2  /* some positions[t] outside [0, rope_rows): that token's rows were not rotated */
#define MLA_STATUS_LEN_RANGE  8  /* mla_latent_gather_launch, mla_prefix_attend_launch: a length, an offset or a position
                                    outside its block table, or group offsets that do not ascend: cut to what the
                                    table holds, or the row left out */
#define MLA_STATUS_TIMEOUT    4  /* a bounded wait inside a kernel (on a copy, a barrier or the tensor cores)
                                    ran out: the outputs are incomplete (mla_prefix_attend_launch: the rows
                                    concerned are NaN).  No such wait is expected ever to run out; the kernel
                                    returns instead of hanging */

/* Kernel choice (mla_plan.mode). */
#define MLA_MODE_SPLIT 1 /* small T: three warps per 576-wide row (two move 16-byte nope chunks, one rotates the
                            32 RoPE pairs, one per lane); rows_per_block rows per block, ceil(rows / SMs) up to 4
                            unless tuned, so a single token's rows run one per SM */
#define MLA_MODE_ROWS  2 /* large T: grid-stride over rows, grid sized to the resident blocks; one warp per row
                            (bf16 outputs) or half a warp per row (an e4m3 output) */

/*
 * mla_epilogue_launch -- the whole epilogue in one kernel launch.
 *
 *   q_nope   bf16 [T, H, 512] at element strides (q_nope_stride_t, q_nope_stride_h, 1)
 *   q_pe     bf16 [T, H, 64]  at (q_pe_stride_t, q_pe_stride_h, 1)
 *   kv_c     bf16 [T, 512]    at (kv_c_stride_t, 1)
 *   k_pe     bf16 [T, 64]     at (k_pe_stride_t, 1)
 *   slot_mapping  int64 [T]: cache row (block * block_size + offset) for token t.
 *            A negative slot skips that token's cache row silently; a slot
 *            >= num_blocks*block_size skips it and sets MLA_STATUS_SLOT_RANGE.
 *            Two tokens with the same slot: which row lands is unspecified.
 *   positions int32 [T] and cos_sin fp32 [rope_rows, 64] (row p = cos_0..31 |
 *            sin_0..31 at position p): read only with MLA_FLAG_ROPE (may be
 *            NULL otherwise).  One position per token, shared by its H query
 *            rows and its cache row.  A position outside [0, rope_rows) leaves
 *            that token's rows unrotated and sets MLA_STATUS_POS_RANGE.
 *   q_scale, kv_scale  one fp32 each in device memory (read by the kernel, so
 *            an upstream kernel may write them); read only with the matching
 *            FP8 flag (may be NULL otherwise).  For any scale the e4m3
 *            byte is that of the IEEE fp32 quotient x / scale (the kernel
 *            computes that quotient bit for bit whenever |x| >= 2^-100 and
 *            |x / scale| < 448; outside, both round to the same signed
 *            zero or to +-448).
 *   T >= 0 tokens (T == 0: nothing is launched, MLA_OK); H >= 1 heads;
 *   block_size >= 1, num_blocks >= 0: cache geometry.
 *   q_out    [T, H, 576] contiguous; bf16, or e4m3 bytes with MLA_FLAG_Q_FP8.
 *   cache    [num_blocks, block_size, 576] contiguous; bf16, or e4m3 bytes with
 *            MLA_FLAG_KV_FP8.  Only the T addressed rows are written; every
 *            other byte is left as it was.
 *   status   optional int32 in device memory (NULL = no reporting); the kernel
 *            ORs MLA_STATUS_* bits into it and never clears it.
 *
 * Alignment (the 16-byte row rule of the vLLM PR #54565 report, section 实现拆解
 * item 1): q_nope, kv_c, q_out and cache start on 16-byte boundaries and the
 * strides of q_nope and kv_c are multiples of 8 elements (a stride is not
 * checked when its dimension has size 1); q_pe and k_pe need only bf16
 * (2-byte) alignment; slot_mapping 8 bytes; positions, cos_sin, scales and
 * status 4 bytes.  Strides must be >= 0.  Otherwise MLA_ERR_ALIGNMENT or
 * MLA_ERR_INVALID_ARG and nothing is launched.  Sizes: H <= 65536 and
 * T * (H + 1) < 2^31.  With q_pe and k_pe rows 4-byte aligned (even strides)
 * and cos_sin 8-byte aligned, MLA_MODE_ROWS with an e4m3 output reads and
 * writes the pe values as vectors; the results are the same either way.
 *
 * Programmatic dependent launch (MLA_FLAG_PDL, as the enable_pdl argument of
 * the vLLM PR #54565 report's GEMM entry): the kernel may start before the
 * previous kernel on `stream` has finished.  Query rows wait for it
 * (griddepcontrol.wait) only right before reading q_nope / q_pe; cache rows,
 * slot_mapping, positions, cos_sin and the scales are read without waiting
 * (PR #54896 report, 实现拆解 item 2).  CONTRACT: with this flag the previous
 * kernel on `stream` may write q_nope and q_pe only, and must not read q_out
 * or the cache rows this call writes (cache rows are written while that
 * kernel may still be running).  The kernel signals its own
 * dependents (griddepcontrol.launch_dependents) only after all of its stores
 * (PR #54896 report, 评论区精华: the early trigger was a race and was moved
 * back to the end).
 */
MLA_API mla_status mla_epilogue_launch(
    const void* q_nope, int64_t q_nope_stride_t, int64_t q_nope_stride_h,
    const void* q_pe, int64_t q_pe_stride_t, int64_t q_pe_stride_h,
    const void* kv_c, int64_t kv_c_stride_t,
    const void* k_pe, int64_t k_pe_stride_t,
    const int64_t* slot_mapping,
    const int32_t* positions,
    const float* cos_sin, int64_t rope_rows,
    const float* q_scale, const float* kv_scale,
    int64_t T, int64_t H, int64_t block_size, int64_t num_blocks,
    uint32_t flags,
    void* q_out,
    void* cache,
    int32_t* status,
    mla_stream_t stream);

/*
 * mla_plan -- the launch mla_epilogue_launch would make for (T, H, flags) on
 * the current device, without launching anything.  Host only; needs the
 * device's SM count, which it reads once per device (sm_count <= 0 lets the
 * caller pass it instead: `sm_count` > 0 is used as given and no CUDA call is
 * made).  Returns MLA_ERR_INVALID_ARG for T < 1, H < 1 or both FORCE flags.
 */
typedef struct mla_plan {
  int32_t mode;              /* MLA_MODE_SPLIT or MLA_MODE_ROWS */
  int32_t threads_per_block;
  int64_t blocks;
  int32_t rows_per_block;    /* SPLIT: rows one block covers (96 threads each); ROWS: rows one warp converts at
                                a time (1, or 2 with an e4m3 output) */
  int32_t sm_count;
} mla_plan;

MLA_API mla_status mla_epilogue_plan(int64_t T, int64_t H, uint32_t flags, int32_t sm_count, mla_plan* out);

/*
 * Tuning knobs of the plan (process-wide; not synchronised, set them before
 * launching from several threads).  The pages choose the small-batch split
 * for up to 64 tokens and note that the threshold may not suit other batch
 * sizes or hardware (PR #54896 report, 风险与影响 "risks" item 2).  On B200
 * the split kernel stays faster than the rows kernel up to about 4.6 K rows
 * (T * (H + 1)) whatever H is (measured for H = 8, 16, 32, 128), so the
 * default threshold counts rows, not tokens.
 *   split_max_rows       T * (H + 1) at or below which MLA_MODE_SPLIT is used (default 4608)
 *   split_rows_per_block rows per block in MLA_MODE_SPLIT (block = 96 * this), at most
 *                        10; 0 (default) takes ceil(rows / SMs), at most 4; a negative
 *                        value restores the default
 *   rows_warps_per_block warps per block in MLA_MODE_ROWS, at most 8 (default 8)
 *   rows_blocks_per_sm   blocks per SM the MLA_MODE_ROWS grid is sized for, at most
 *                        the number the kernel's register cap keeps resident (4 with
 *                        an e4m3 output, 5 without; default: that number)
 * Larger values are clamped to those limits; 0 keeps the current setting.
 */
typedef struct mla_tuning {
  int64_t split_max_rows;
  int32_t split_rows_per_block;
  int32_t rows_warps_per_block;
  int32_t rows_blocks_per_sm;
} mla_tuning;

MLA_API void mla_epilogue_set_tuning(const mla_tuning* t);
MLA_API void mla_epilogue_get_tuning(mla_tuning* out);

/* ======================================================================================
 * Latent cache rows: writing with a norm and microscaled codes, reading back, attending.
 *
 * Formats of a cache row (`format` of the entry points below):
 *   MLA_CACHE_BF16  576 bf16 values (1152 bytes), as mla_epilogue_launch writes;
 *   MLA_CACHE_E4M3  576 e4m3 bytes, value = code * *kv_scale, as mla_epilogue_launch
 *                   writes with MLA_FLAG_KV_FP8;
 *   MLA_CACHE_MX    656 bytes: 512 e4m3 codes of the latents, then 16 scale bytes, one
 *                   for each 32 latents (value = code * 2^(byte - 127)), then the 64
 *                   rotary values in bf16 (at byte 528).
 * ====================================================================================== */
#define MLA_CACHE_BF16 0
#define MLA_CACHE_E4M3 1
#define MLA_CACHE_MX   2

/*
 * mla_latent_insert_launch -- one latent cache row per token, with the norm of
 * the latents, the rotation and the quantisation in the same pass:
 *
 *   y  = kv_c[t] * rsqrt(mean(kv_c[t]^2) + eps) * norm_weight   (norm_weight NULL: y = kv_c[t])
 *   pe = rope(k_pe[t]) with MLA_FLAG_ROPE, else k_pe[t]
 *   cache.row(slot_mapping[t]) = encode(y || pe)
 *
 * y is computed in 64 bits and rounded once to fp32; rope and its table are
 * those of mla_epilogue_launch (fp32, every operation rounded).  encode:
 *   MLA_CACHE_BF16  bf16, ties to even;
 *   MLA_CACHE_E4M3  e4m3 of the IEEE fp32 quotient x / *kv_scale, ties to even,
 *                   saturating at +-448 (infinities too), NaN stays NaN;
 *   MLA_CACHE_MX    per 32 latents e = the least integer with max |y| <= 448 * 2^e
 *                   over the finite y, kept within [-117, 119] (-117 for a group of
 *                   zeros); code = e4m3 of y * 2^-e as above, scale byte = e + 127;
 *                   pe in bf16.  Only a value beyond 448 * 2^119 or an infinity
 *                   saturates; y below 2^-10 * 2^-117 may become zero.
 *
 *   kv_c   bf16 [T, 512] at (kv_c_stride_t, 1), 16-byte aligned, stride a multiple of
 *          8 (unchecked for T == 1); k_pe bf16 [T, 64] at (k_pe_stride_t, 1)
 *   slot_mapping, positions, cos_sin, rope_rows, kv_scale, status: as in
 *          mla_epilogue_launch; kv_scale is read with MLA_CACHE_E4M3 only
 *   norm_weight  bf16 [512], 16-byte aligned, or NULL; eps >= 0 (finite)
 *   cache  [num_blocks, block_size, row] contiguous, 16-byte aligned
 *   flags  MLA_FLAG_ROPE, MLA_FLAG_PDL (CONTRACT: the previous kernel on `stream` may
 *          write kv_c and k_pe only; everything else is read before waiting for it,
 *          and the cache rows are written after)
 * T >= 0, T < 2^31.  A token whose slot is negative or out of range writes nothing.
 */
MLA_API mla_status mla_latent_insert_launch(
    const void* kv_c, int64_t kv_c_stride_t,
    const void* k_pe, int64_t k_pe_stride_t,
    const int64_t* slot_mapping,
    const void* norm_weight, float eps,
    const int32_t* positions, const float* cos_sin, int64_t rope_rows,
    const float* kv_scale,
    int64_t T, int64_t block_size, int64_t num_blocks,
    int32_t format, uint32_t flags,
    void* cache, int32_t* status, mla_stream_t stream);

/*
 * mla_latent_gather_launch -- rows of paged sequences read back as bf16:
 *
 *   for b < B, cu_rows[b] <= r < cu_rows[b+1], r < N:   k = first[b] + r - cu_rows[b]
 *     out[r] = bf16(decode(cache.row(block_table[b][k / block_size] * block_size + k % block_size)))
 *
 * decode: bf16 rows are copied bit for bit; e4m3 is the fp32 product
 * code * *kv_scale rounded to bf16; a microscaled value is exact in bf16.
 *   block_table int32 [B, table_cols] at row stride table_stride (elements)
 *   cu_rows     int32 [B + 1], ascending; rows r >= cu_rows[B] of out stay as they were
 *   first       int32 [B] or NULL (0): position each sequence is read from
 *   out         bf16 [N, 576] at row stride out_stride (a multiple of 8), 16-byte aligned
 * A page number outside [0, num_blocks) sets MLA_STATUS_SLOT_RANGE, a position
 * outside the table MLA_STATUS_LEN_RANGE; such a row of out stays as it was.
 * B >= 0, N >= 0, both < 2^31.  flags: MLA_FLAG_PDL (everything is read after the wait).
 */
MLA_API mla_status mla_latent_gather_launch(
    const void* cache, int32_t format, int64_t block_size, int64_t num_blocks, const float* kv_scale,
    const int32_t* block_table, int64_t table_stride, int64_t table_cols,
    const int32_t* cu_rows, const int32_t* first, int64_t B, int64_t N,
    uint32_t flags, void* out, int64_t out_stride, int32_t* status, mla_stream_t stream);

/*
 * mla_prefix_attend_launch -- decode attention over the paged latent cache for a
 * batch whose tokens share long prefixes.  Token t of group g (group_offsets[g] <=
 * t < group_offsets[g+1]) attends to the prefix_lens[g] keys in the pages
 * prefix_table[g] and then to its own seq_lens[t] keys in block_table[t]:
 *
 *   s[t, h, k]  = sm_scale * sum_d q[t, h, d] * key[k, d]            d < 576
 *   lse[t, h]   = log sum_k exp(s[t, h, k])
 *   out[t, h, d] = sum_k exp(s[t, h, k] - lse[t, h]) * key[k, d]     d < 512
 *
 * key[k] is the decoded cache row and q the decoded query (e4m3 code * *q_scale
 * with MLA_FLAG_Q_FP8).  The keys of a prefix are read and multiplied once for
 * all rows (token, head) of its group, 64 rows at a time.  A row with no keys
 * gets out = 0 and lse = -inf.  Tokens before group_offsets[0] or from
 * group_offsets[G] on have no prefix.
 *
 * Products run on the tensor cores with fp32 accumulation; scores, softmax
 * statistics and partial sums are fp32; the softmax weights are rounded to bf16
 * before they multiply the keys.  When both q and the cache are e4m3, the codes
 * themselves are multiplied, and a weight is the sum of three e5m2 numbers (nine
 * bits, one more than bf16's; with scores below 2^21, what weights too small for
 * that lose is together at most 2^-11 of the denominator, or 2^-30 for each key of a
 * token where those are more).  A product of q and a key beyond fp32's range is an
 * infinity, and a row whose largest score is one comes out as NaN.  So may a row
 * whose largest score is beyond 2^30 in magnitude, or 2^27 with q and cache in e4m3.
 *
 *   q       [T, H, 576] at element strides (q_stride_t, q_stride_h, 1): bf16, or e4m3
 *           bytes with MLA_FLAG_Q_FP8; 16-byte aligned, strides multiples of 16 bytes
 *           (unchecked for a size-1 dimension), >= 0
 *   cache, format, block_size, num_blocks, kv_scale: as above
 *   prefix_table int32 [G, prefix_cols] at row stride prefix_stride; prefix_lens int32 [G];
 *           group_offsets int32 [G + 1], ascending (NULL with G == 1: every token).
 *           G == 0: no prefixes, all three NULL
 *   block_table int32 [T, table_cols] at row stride table_stride; seq_lens int32 [T].
 *           table_cols == 0 (block_table NULL): no token has keys of its own
 *   out     bf16 [T, H, 512] contiguous, 16-byte aligned;  lse fp32 [T, H] or NULL
 *   workspace  mla_prefix_attend_workspace_for() bytes (prefix_keys = prefix_cols *
 *           block_size; sm_count 0: of the current device) of device memory, 256-byte
 *           aligned; mla_prefix_attend_workspace() bytes are enough for every cache.
 *           Groups of 256 rows or more on average, over a cache that needs decoding or
 *           has odd pages, take up to 73856 bytes for each 64 keys of prefix_keys, 2 GiB
 *           at most.  Need not be initialised, holds nothing between calls; two calls
 *           that may run at the same time need two
 *   flags   MLA_FLAG_Q_FP8, MLA_FLAG_PDL (everything is read after the wait)
 * A negative length counts as 0.  A length beyond its table is cut to it and sets
 * MLA_STATUS_LEN_RANGE.  Keys in a page outside [0, num_blocks) are left out and
 * set MLA_STATUS_SLOT_RANGE.  Keys behind a sequence's length are never read.
 * T >= 0, 1 <= H <= 65535, T * H < 2^31 - 64, 0 <= G <= T.
 */
MLA_API mla_status mla_prefix_attend_workspace(int64_t T, int64_t H, int64_t G, int64_t prefix_keys, int32_t sm_count,
                                               int64_t* bytes);
MLA_API mla_status mla_prefix_attend_workspace_for(int64_t T, int64_t H, int64_t G, int64_t prefix_keys, int32_t format,
                                                   uint32_t flags, int64_t block_size, int64_t num_blocks,
                                                   int32_t sm_count, int64_t* bytes);

MLA_API mla_status mla_prefix_attend_launch(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const float* q_scale,
    const void* cache, int32_t format, int64_t block_size, int64_t num_blocks, const float* kv_scale,
    const int32_t* prefix_table, int64_t prefix_stride, int64_t prefix_cols,
    const int32_t* prefix_lens, const int32_t* group_offsets, int64_t G,
    const int32_t* block_table, int64_t table_stride, int64_t table_cols, const int32_t* seq_lens,
    int64_t T, int64_t H, float sm_scale, uint32_t flags,
    void* out, float* lse, void* workspace, int64_t workspace_bytes, int32_t* status, mla_stream_t stream);

/* Text for a status code (static storage). */
MLA_API const char* mla_status_string(mla_status s);

/* The cudaError_t of the last launch that returned MLA_ERR_CUDA on this host thread (0 if none). */
MLA_API int32_t mla_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_EPILOGUE_H */
