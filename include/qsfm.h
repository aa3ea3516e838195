/*
 * qsfm.h — C ABI of the quantized shared-KV sparse MLA attention forward
 * (QuantSparseFlashMla / KvQuantSparseAttnSharedKv) for sm_103a.
 *
 * What is computed (QuantSparseFlashMla, "功能说明" (function description),
 * formula O = softmax(Q K~^T * softmax_scale) V~ with K~ = V~; the per-head
 * sink is the "sinks" row of its "参数说明" (parameter) table):
 *
 *   for every query token t (batch b, position s) and head h (N1 = 64 or
 *   128 heads, D = 512, one latent KV head, N2 = 1):
 *     rows(t) = ori rows inside the band / causal window of t
 *             ++ cmp rows (CSA: the valid entries of cmp_sparse_indices[t];
 *                          HCA: every causally visible compressed row)
 *     K~[j, d] = e4m3fn(kv[j, d]) * scale[j, d / 64]
 *     x_j      = softmax_scale * sum_d Q[t, h, d] K~[j, d]
 *     O[t, h]  = sum_j e^{x_j} K~[j, :] / (sum_j e^{x_j} + e^{sink_h})
 *     lse[t,h] = log sum_j e^{x_j}          (the sink is not included)
 *   A token with no attended row gets O = 0 and lse = -inf. A NaN in an attended
 *   row makes the token's O and lse NaN, one in a head's query those of the head
 *   (fp8 rows: a query that is not finite takes the scale that the 64 heads of its
 *   group share in f16, so that the other heads' O and lse are not to be used).
 *
 * Modes (QuantSparseFlashMla, "约束说明" (constraints), third bullet):
 *   SWA  cmp_kv == NULL                        ori window only
 *   CSA  cmp_kv != NULL, cmp_sparse_indices    window + top-k compressed rows
 *   HCA  cmp_kv != NULL, indices == NULL       window + all visible cmp rows
 *
 * Data layout (all device memory is owned by the caller; the library never
 * allocates, frees or keeps pointers after a call returns):
 *   q            bf16  BSND [B, S1, N1, 512] or TND [T1, N1, 512]
 *   attn_out     bf16  same shape as q
 *   softmax_lse  fp32  BSND [B, 1, S1, N1] / TND [1, T1, N1]
 *                      (KvQuantSparseAttnSharedKv, parameter table, row
 *                      softmax_lse); element (token t, head h) at t*N1 + h
 *   ori_kv       fp8 e4m3fn, paged [ori_num_blocks, 128, 1, 512]
 *   cmp_kv       fp8 e4m3fn, paged [cmp_num_blocks, 128, 1, 512]
 *   ori_scale / cmp_scale
 *                fp32 [num_blocks, 128, 1, 8]: one dequant scale per
 *                64-element tile of a row, paged exactly like its KV
 *                (KvQuantSparseAttnSharedKv, parameter table, rows
 *                kv_quant_mode and tile_size: per-tile quantisation, tile 64)
 *   *_block_table int32 [B, *_max_blocks]: logical block -> physical block
 *                (QuantSparseFlashMla, "约束说明", PageAttention bullets)
 *   non-paged KV (layout_kv BSND / TND, QuantSparseFlashMla "约束说明" on
 *   layout_kv): ori_kv [B, S2, 1, row] / [T2, 1, row] and cmp_kv
 *                [B, S3, 1, row] / [T3, 1, row], scales [.., 8] alike;
 *                batch b's row j is at [b, j] (BSND) or at
 *                cu_seqlens_ori_kv[b] + j / cu_seqlens_cmp_kv[b] + j (TND);
 *                no block tables
 *   ori_sparse_indices int32 BSND [B, S1, 1, K1] / TND [T1, 1, K1] or NULL:
 *                discrete picks of ori rows (a logical ori row of the
 *                token's batch; -1 = invalid). When given they replace the
 *                contiguous ori range: the token attends the entries (the
 *                first ori_topk_length[t] when that is given) that lie in
 *                its ori mask range, each occurrence once, in index order
 *   cmp_sparse_indices int32 BSND [B, S1, 1, K2] / TND [T1, 1, K2];
 *                an entry is a logical compressed-row index of the token's
 *                own batch; -1 (or any value outside the visible range) is
 *                ignored
 *   cu_seqlens_q int32 [B + 1], prefix sums from 0 (required for TND)
 *   seqused_q    int32 [B] or NULL (BSND: rows s >= seqused_q[b] are
 *                padding; they get O = 0, lse = -inf)
 *   seqused_ori_kv int32 [B]: ori length S2 of each batch. Required for
 *                paged KV; optional for BSND KV (default: the S2
 *                dimension); must be NULL for TND KV (S2 = cu_seqlens_ori_kv
 *                difference)
 *   seqused_cmp_kv int32 [B] or NULL (default: floor(S2 / cmp_ratio) for
 *                paged KV, the S3 dimension for BSND KV, the
 *                cu_seqlens_cmp_kv difference for TND KV)
 *   cmp_residual_kv int32 [B] or NULL (default 0), 0 <= r_b < cmp_ratio
 *   cmp_topk_length int32 [T] or NULL: only the first n entries of the
 *                token's index row are read
 *   sinks        fp32 [N1] or NULL (NULL: no sink)
 *   metadata     int32 [1024] written by qsfm_metadata()
 *
 * Query position alignment is bottom-right: p = S2 - S1_b + s on the ori
 * side and p_c = cmp_len * cmp_ratio + residual - S1_b + s on the cmp side.
 * ori mask mode 4 (band) keeps rows max(0, p - wl) .. min(S2 - 1, p + wr),
 * -1 meaning no bound on that side; mode 3 keeps rows <= p; mode 0 keeps all.
 * cmp mask mode 3 keeps compressed rows c < floor((p_c + 1) / cmp_ratio)
 * (clipped to [0, cmp_len]); mode 0 keeps all cmp_len rows.
 *
 * Every call is asynchronous on the given stream and never reads device
 * memory back to the host, so the calls may be captured in a CUDA graph
 * (QuantSparseFlashMla, "约束说明": aclgraph mode). Argument errors are found
 * on the host before anything is launched and are returned as status codes.
 * Bad device data (a block id outside the pool, a block-table column past
 * its width) is not trapped: the row is skipped and a bit is set in the
 * device fault word, which qsfm_get_device_status() reads.
 */
#ifndef QSFM_H
#define QSFM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QSFM_ABI_VERSION 6
#define QSFM_NUM_HEADS 64
#define QSFM_HEAD_DIM 512
#define QSFM_BLOCK_SIZE 128
#define QSFM_SCALES_PER_ROW 8
#define QSFM_METADATA_INTS 1024
#define QSFM_MAX_CTAS 256
#define QSFM_PACKED_ROW_BYTES 640
#define QSFM_BF16_ROW_BYTES 1024
#define QSFM_PACKED384_ROW_BYTES 384

/* KV row formats (qsfm_params.kv_layout). */
typedef enum {
  /* fp8 e4m3fn rows [blocks, 128, 1, 512] with fp32 scale tensors
   * [blocks, 128, 1, 8], one scale per 64 elements (the default). */
  QSFM_KV_FP8_FP32_SCALES = 0,
  /* Packed 640-byte rows [blocks, 128, 1, 640] (KvQuantSparseAttnSharedKv
   * constraints): bf16 rope (64 elements, bytes 0..127), e4m3fn nope (448
   * elements, bytes 128..575), e8m0 scales (7, one per 64 nope elements,
   * bytes 576..582), zero padding to 640. The 512 elements of a row are
   * rope then nope; ori_scale and cmp_scale must be NULL. */
  QSFM_KV_PACKED640 = 1,
  /* bf16 rows [blocks, 128, 1, 512] without quantisation (the KV of
   * SparseCompressedFlashAttention); ori_scale and cmp_scale must be NULL. */
  QSFM_KV_BF16 = 2,
  /* 4-bit rows [blocks, 128, 1, 384], an addition of this library: bf16
   * rope (64 elements, bytes 0..127), e2m1 nope (448 codes, bytes 128..351,
   * the lower element in the low nibble), e4m3fn scales (28, one per 16
   * nope elements, bytes 352..379), one e8m0 exponent for the row's scales
   * (byte 380), zero padding to 384. The 512 elements of a row are rope then
   * nope; nope element i is code_i * scale_(i / 16) * 2^(exponent - 127),
   * which has at most six significant bits. ori_scale and cmp_scale must be
   * NULL. qsfm_norm_rope_store() writes such rows. */
  QSFM_KV_PACKED384 = 3
} qsfm_kv_layout;

typedef enum {
  QSFM_OK = 0,
  QSFM_ERR_INVALID_ARG = 1,  /* a constraint of the op is violated        */
  QSFM_ERR_UNSUPPORTED = 2,  /* valid for the op but not built             */
  QSFM_ERR_CUDA = 3,         /* a CUDA runtime call failed                */
  QSFM_ERR_WORKSPACE = 4,    /* workspace NULL or smaller than required   */
  QSFM_ERR_DEVICE_FAULT = 5, /* the device fault word is non-zero         */
  QSFM_ERR_TIMEOUT = 6       /* reserved for bounded device waits         */
} qsfm_status;

typedef enum { QSFM_LAYOUT_BSND = 0, QSFM_LAYOUT_TND = 1 } qsfm_q_layout;

/* KV storage (qsfm_params.layout_kv; QuantSparseFlashMla parameter table
 * row layout_kv and its constraints: BSND / TND KV only with the same q
 * layout, paged KV with either). */
typedef enum {
  QSFM_LAYOUT_KV_PA_BBND = 0, /* paged 128-row blocks through block tables  */
  QSFM_LAYOUT_KV_BSND = 1,    /* [B, S, 1, row] per batch slab              */
  QSFM_LAYOUT_KV_TND = 2      /* [T, 1, row], batches at cu_seqlens_*_kv    */
} qsfm_layout_kv;

/* Device fault word bits (qsfm_get_device_status). */
#define QSFM_FAULT_ORI_BLOCK_ID   0x1  /* ori block table entry outside pool */
#define QSFM_FAULT_CMP_BLOCK_ID   0x2  /* cmp block table entry outside pool */
#define QSFM_FAULT_ORI_TABLE_COL  0x4  /* ori row beyond the table width     */
#define QSFM_FAULT_CMP_TABLE_COL  0x8  /* cmp row beyond the table width     */
#define QSFM_FAULT_METADATA       0x10 /* metadata header does not match     */
#define QSFM_FAULT_TIMEOUT        0x20 /* a bounded device wait ran out      */
#define QSFM_FAULT_RANGE          0x40 /* an fp8 KV row dequantises past
                                          2^22: its values were clamped    */
#define QSFM_FAULT_KV_ROW         0x80 /* a non-paged KV row past the end of
                                          its tensor (skipped)             */
#define QSFM_FAULT_BLOCK_POOL     0x100 /* qsfm_update_block_tables(): no free
                                          block was left, or the free list
                                          would have overflowed            */
#define QSFM_FAULT_SLOT           0x200 /* a slot past the end of the cache, or
                                          more new rows than slot_map holds */
#define QSFM_FAULT_POSITION       0x400 /* a position past the cos_sin table */
#define QSFM_FAULT_ROW_INDEX      0x800 /* a row_index past the source rows  */
#define QSFM_FAULT_GROUP_ROWS     0x1000 /* cu_rows that decreases or leaves
                                           the rows of the product           */

/*
 * All inputs, attributes and outputs of one forward call. Pointers are
 * device pointers; NULL marks an absent optional input. q, ori_kv, cmp_kv and
 * attn_out must be 16-byte aligned (packed384 ori_kv and cmp_kv 32-byte
 * aligned) and every other pointer 4-byte aligned
 * (QSFM_ERR_INVALID_ARG otherwise). The parameter names follow
 * QuantSparseFlashMla, "参数说明" (parameter table).
 * Size limits of the kernels' 32-bit index arithmetic (QSFM_ERR_UNSUPPORTED
 * beyond them; every batch that fits in device memory is far below): at
 * most 2^24 work units (tokens x n1 / 64), k2 <= 65536, and fewer than 2^31
 * rows in each KV pool (num_blocks x block_size).
 */
typedef struct qsfm_params {
  /* shapes */
  int32_t batch;          /* B                                               */
  int32_t max_s1;         /* BSND: S1. TND: unused                           */
  int32_t total_t;        /* TND: T1 (= q.shape[0]). BSND: unused            */
  int32_t n1;             /* query heads: 64 or 128 (the pages allow both)   */
  int32_t d;              /* head dim; must be 512                           */
  int32_t k2;             /* index row length K2 (CSA); 0 otherwise          */
  int32_t ori_block_size; /* tokens per ori block; only 128 is built         */
  int32_t cmp_block_size; /* tokens per cmp block; only 128 is built         */
  int32_t ori_max_blocks; /* ori_block_table row width                       */
  int32_t cmp_max_blocks; /* cmp_block_table row width                       */
  int32_t ori_num_blocks; /* physical blocks in the ori pool                 */
  int32_t cmp_num_blocks; /* physical blocks in the cmp pool                 */
  int32_t num_ctas;       /* most CTAs the work is planned over; 0 = SM
                             count. The plan's units are the 64-head groups
                             of the tokens (U = T * n1 / 64). With U >=
                             num_ctas the plan uses ceil(U / ceil(U /
                             num_ctas)) CTAs, the fewest that keep the same
                             units per CTA                                  */
  /* inputs (device) */
  const void* q;
  const void* ori_kv;
  const float* ori_scale;
  const void* cmp_kv;
  const float* cmp_scale;
  const int32_t* cmp_sparse_indices;
  const int32_t* ori_block_table;
  const int32_t* cmp_block_table;
  const int32_t* cu_seqlens_q;
  const int32_t* seqused_q;
  const int32_t* seqused_ori_kv;
  const int32_t* seqused_cmp_kv;
  const int32_t* cmp_residual_kv;
  const int32_t* cmp_topk_length;
  const float* sinks;
  const int32_t* metadata;
  /* attributes */
  float softmax_scale;
  int32_t cmp_ratio;      /* 1..128; must be 1 when cmp_kv is NULL           */
  int32_t ori_mask_mode;  /* 0, 3 or 4                                       */
  int32_t cmp_mask_mode;  /* 0 or 3                                          */
  int32_t ori_win_left;   /* -1 or >= 0; >= 0 only with ori_mask_mode 4      */
  int32_t ori_win_right;  /* -1 or >= 0; >= 0 only with ori_mask_mode 4      */
  int32_t layout_q;       /* qsfm_q_layout                                   */
  int32_t return_lse;     /* non-zero: write softmax_lse                     */
  /* outputs (device) */
  void* attn_out;
  float* softmax_lse;
  /* appended in ABI version 2 */
  int32_t kv_layout;      /* qsfm_kv_layout of ori_kv and cmp_kv (both)      */
  /* appended in ABI version 3 */
  int32_t layout_kv;      /* qsfm_layout_kv of ori_kv and cmp_kv (both)      */
  int32_t ori_kv_len;     /* BSND / TND KV: length of ori_kv's sequence axis
                             (S2 of [B, S2, 1, row], T2 of [T2, 1, row])     */
  int32_t cmp_kv_len;     /* the same for cmp_kv (S3 / T3)                   */
  int32_t k1;             /* ori_sparse_indices row length K1; 0 without     */
  const int32_t* cu_seqlens_ori_kv;  /* int32 [B + 1]: TND KV (required)      */
  const int32_t* cu_seqlens_cmp_kv;  /* int32 [B + 1]: TND KV with cmp_kv    */
  const int32_t* ori_sparse_indices; /* see the data layout above            */
  const int32_t* ori_topk_length;    /* int32 [T] or NULL: entries of the
                                        token's ori index row that count    */
} qsfm_params;

/* Fill *p with the defaults of the op: n1 64, d 512, block size 128,
 * cmp_ratio 1, ori mask 4 with window 127/0 (KvQuantSparseAttnSharedKv,
 * parameter table rows ori_mask_mode, ori_win_left, ori_win_right), cmp mask
 * 3, softmax_scale 1/sqrt(512), layout BSND, all pointers NULL. */
void qsfm_params_init(qsfm_params* p);

/*
 * Plan the work of one forward call over p->num_ctas CTAs (the split-core
 * plan of QuantSparseFlashMlaMetadata, QuantSparseFlashMla "功能说明",
 * calling sequence steps 1-3). Reads cu_seqlens_q / seqused_* /
 * cmp_residual_kv / cmp_topk_length on the device and writes the int32[1024]
 * plan to metadata_out (device memory, caller-owned). Launches one small
 * kernel on `stream`; nothing is read back.
 * Errors: QSFM_ERR_INVALID_ARG for a NULL metadata_out or invalid params.
 */
qsfm_status qsfm_metadata(const qsfm_params* p, int32_t* metadata_out,
                          void* stream /* cudaStream_t */);

/* Bytes of device workspace qsfm_forward() needs for p (partial outputs of
 * work split across CTAs). May be 0. */
qsfm_status qsfm_forward_workspace_size(const qsfm_params* p, size_t* bytes);

/*
 * The forward pass: attention kernel, then (only when the plan may split a
 * token across CTAs) the log-sum-exp combine kernel. Writes attn_out and,
 * when return_lse is set, softmax_lse. p->metadata must come from
 * qsfm_metadata() with the same shapes and lengths (QuantSparseFlashMla,
 * "约束说明": metadata is required, shape [1024]). A call gives the same bits
 * every time. In another batch a token may differ in its last bits: where it is
 * split otherwise, and over 4-bit rows also by the tokens worked on before it,
 * whose maxima are the first reference of its softmax.
 * workspace: device memory of at least qsfm_forward_workspace_size() bytes.
 */
qsfm_status qsfm_forward(const qsfm_params* p, void* workspace,
                         size_t workspace_bytes, void* stream);

/* The two stages of qsfm_forward(), callable separately (for timing). */
qsfm_status qsfm_attention(const qsfm_params* p, void* workspace,
                           size_t workspace_bytes, void* stream);
qsfm_status qsfm_combine(const qsfm_params* p, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * qsfm_forward() for callers that cannot allocate device memory. The paper
 * has no counterpart: this is an addition of this library.
 *
 * Some callers cannot call cudaMalloc: code that runs inside another
 * framework's memory pool, plugin hosts that hand over only the input and
 * output buffers, serving loops that forbid allocation once running. This
 * entry point allocates nothing. Instead of a workspace argument it uses a
 * fixed scratch array of QSFM_NOALLOC_SCRATCH_BYTES that the library
 * reserves in the memory of every GPU that loads it, held until the process
 * exits. The caller still passes all inputs and outputs (and the metadata
 * from qsfm_metadata()) in p.
 *   - Returns QSFM_ERR_WORKSPACE, launching nothing, when the plan needs
 *     more than QSFM_NOALLOC_SCRATCH_BYTES of partial results (that happens
 *     only when tokens may be split over CTAs, i.e. fewer query tokens than
 *     p->num_ctas; the need is 2 * num_ctas * 131328 bytes rounded up, so at
 *     most 31 CTAs fit). qsfm_forward_workspace_size() gives the need.
 *   - The first call on a device looks up the array's device address with
 *     that device current; make it before any stream capture.
 *   - All calls share the array, which keeps the last call's contents;
 *     nothing in it needs to start at zero. Calls that overlap on the GPU
 *     (other streams or threads) race on it.
 */
#define QSFM_NOALLOC_SCRATCH_BYTES (8u << 20)
qsfm_status qsfm_forward_noalloc(const qsfm_params* p, void* stream);

/*
 * Debug export of the row resolution the attention kernel uses. For each
 * of the n query tokens in tokens[] (device int32), writes the token's row
 * slots in the kernel's order (ori window rows, then cmp slots), up to
 * max_rows of them:
 *   rows_out    uint8 [n, max_rows, R]    the bytes of the resolved row in
 *                                         the pool's own format, R = 512
 *                                         (fp8), 640 or 384 (packed) or 1024
 *                                         (bf16)
 *   scales_out  fp32  [n, max_rows, 8]    its dequant scales (fp8 only)
 *   row_ids_out int32 [n, max_rows]       (source << 30) | logical row, with
 *                                         source 0 = ori, 1 = cmp; -1 for a
 *                                         slot that is masked out
 *   counts_out  int32 [n]                 number of slots of the token
 * Masked slots get zero bytes and zero scales. All buffers are device memory
 * and rows_out must be 16-byte aligned. rows_out and scales_out may both be
 * NULL: then only the row ids and counts are written. For the fp8 format
 * rows_out and scales_out are given together or not at all; for the others
 * scales_out must be NULL (QSFM_ERR_INVALID_ARG otherwise). row_ids_out is
 * required when max_rows > 0.
 */
qsfm_status qsfm_debug_gather(const qsfm_params* p, const int32_t* tokens,
                              int32_t n, int32_t max_rows, uint8_t* rows_out,
                              float* scales_out, int32_t* row_ids_out,
                              int32_t* counts_out, void* stream);

/*
 * Debug check of the bounded waits every kernel of the library uses (no GPU
 * fault, no hang). One block: a thread waits with a limit of timeout_ns on
 * an mbarrier that nothing arrives on; when the limit runs out it raises the
 * block's abort flag and sets QSFM_FAULT_TIMEOUT in the fault word. A thread
 * of another warp waits on a second such barrier with a limit 1000 times as
 * long and gives up as soon as it sees the abort flag. Writes the two waits'
 * durations in ns to elapsed_ns_out[0..1] (device memory, caller-owned).
 * Errors: QSFM_ERR_INVALID_ARG for a NULL output, or timeout_ns of 0 or
 * above one second.
 */
qsfm_status qsfm_debug_bounded_wait(uint64_t timeout_ns, uint64_t* elapsed_ns_out, void* stream);

/*
 * Lightning-indexer top-k (QuantLightningIndexerV2, "功能说明" formula and
 * "参数说明" (parameter table); quant mode 1: FLOAT8_e4m3fn query and key,
 * fp32 dequant scales and weights). For every query token t (batch b,
 * position s) and every key j it may see:
 *   score_j = sum_h weights[t, h] * ReLU(query_scale[t, h] * key_scale[j]
 *                                        * sum_d query[t, h, d] key[j, d])
 * and sparse_indices[t] lists the topk keys of largest score (the smaller
 * key index first among equal scores) in ascending key order, then -1 up
 * to topk (valid entries first, -1 after, as KvQuantSparseAttnSharedKv's
 * constraints want of an index row). Keys visible to the token: all
 * j < seqused_k[b] (mask_mode 0), or only j < floor((p_c + 1) / cmp_ratio)
 * with p_c = seqused_k[b] * cmp_ratio + cmp_residual_k[b] - S1_b + s
 * (mask_mode 3, the compressed rows' right-down-causal rule). A padded
 * query row (seqused_q) gets -1 everywhere.
 *
 * Layout (all device memory, caller-owned):
 *   query        e4m3fn bytes BSND [B, S1, heads, dim] / TND [T, heads, dim]
 *   query_scale  fp32 [T, heads];  weights fp32 [T, heads]
 *   key          e4m3fn bytes (parameter table: layout_k):
 *                  PA_BBND (default) paged [num_blocks, 128, 1, dim] through
 *                    block_table int32 [B, max_blocks], seqused_k[b] keys
 *                    (seqused_k required);
 *                  BSND [B, max_sk, 1, dim], batch b's key j at [b, j],
 *                    seqused_k[b] keys (max_sk when seqused_k is NULL);
 *                  TND [total_k, 1, dim], batch b's key j at row
 *                    cu_seqlens_k[b] + j, cu_seqlens_k[b + 1] - cu_seqlens_k[b]
 *                    keys (cu_seqlens_k int32 [B + 1] required, seqused_k
 *                    NULL)
 *   key_scale    fp32, the key's layout without the dim axis
 *   output_idx_offset int32 [B] or NULL: every valid index of a batch-b row
 *                is reported plus output_idx_offset[b] (-1 stays -1)
 *   cmp_residual_k int32 [B] or NULL (0);  cu_seqlens_q int32 [B + 1]
 *                (required for TND);  seqused_q int32 [B] or NULL: query
 *                rows of batch b from seqused_q[b] on are padding (all -1;
 *                the other rows keep their positions, S1_b being the chunk
 *                length of the layout), for BSND and TND alike
 *   sparse_indices int32 [T, 1, topk] (out)
 *   sparse_values  bf16 [T, 1, topk] (out, written when return_value != 0;
 *                the scores of the listed keys, -inf after them)
 * Built shapes (QSFM_ERR_UNSUPPORTED otherwise): dim = 128, 1 <= heads
 * <= 64, 1 <= topk <= 8192, block size 128, at most 2^20 query rows, at
 * most 32768 keys per batch and at most max_blocks * 128 (paged) or max_sk
 * (BSND) of them; a larger key count is cut and flagged
 * (QSFM_FAULT_KV_ROW past 32768 or past the end of a TND key tensor, else
 * QSFM_FAULT_CMP_TABLE_COL). A block id outside [0, num_blocks) is flagged
 * with QSFM_FAULT_CMP_BLOCK_ID, its keys score -inf and are not read.
 * Pointers: query, key, key_scale 16-byte aligned, the rest 4-byte aligned.
 */
typedef struct qsfm_indexer_params {
  int32_t batch;        /* B                                                */
  int32_t max_s1;       /* BSND: S1                                         */
  int32_t total_t;      /* TND: T (query rows)                              */
  int32_t heads;        /* g, query heads of the indexer                    */
  int32_t dim;          /* d, must be 128                                   */
  int32_t topk;         /* 1 .. 8192                                        */
  int32_t block_size;   /* keys per block; only 128 is built                */
  int32_t max_blocks;   /* block_table row width                            */
  int32_t num_blocks;   /* blocks in the key pool                           */
  int32_t layout_q;     /* qsfm_q_layout                                    */
  int32_t mask_mode;    /* 0 or 3                                           */
  int32_t cmp_ratio;    /* 1 .. 128                                         */
  int32_t return_value; /* non-zero: write sparse_values                    */
  const void* query;
  const float* query_scale;
  const float* weights;
  const void* key;
  const float* key_scale;
  const int32_t* block_table;
  const int32_t* seqused_k;
  const int32_t* cmp_residual_k;
  const int32_t* cu_seqlens_q;
  const int32_t* seqused_q;
  int32_t* sparse_indices;
  void* sparse_values;
  /* version 6: the key layouts and the index offset */
  int32_t layout_k;     /* qsfm_kv_layout: PA_BBND (default), BSND or TND   */
  int32_t max_sk;       /* BSND keys: S_k, the key tensor's S dimension     */
  int32_t total_k;      /* TND keys: T_k, the key tensor's rows             */
  const int32_t* cu_seqlens_k;
  const int32_t* output_idx_offset;
} qsfm_indexer_params;

/* Defaults: dim 128, heads 64, topk 2048 (the page's default), block size
 * 128, mask_mode 0, cmp_ratio 1, layout BSND, all pointers NULL. */
void qsfm_indexer_params_init(qsfm_indexer_params* p);

/* Bytes of device workspace qsfm_lightning_indexer() needs for p: one fp32
 * score row of min(32768, max_blocks * 128) entries per query row. Reads
 * no device memory. Errors as qsfm_lightning_indexer() for the attributes. */
qsfm_status qsfm_lightning_indexer_workspace_size(const qsfm_indexer_params* p, size_t* bytes);

/* The indexer's top-k: a score kernel writes every visible key's score into
 * the workspace, a select kernel then lists each row's top-k. workspace:
 * caller-owned device memory, 16-byte aligned, of at least
 * qsfm_lightning_indexer_workspace_size() bytes, not read before it is
 * written. Asynchronous on `stream`, no allocation, nothing read back.
 * Errors: QSFM_ERR_INVALID_ARG (missing or misaligned pointers, bad
 * attributes), QSFM_ERR_UNSUPPORTED (shapes not built), QSFM_ERR_WORKSPACE
 * (workspace NULL, misaligned or too small). */
qsfm_status qsfm_lightning_indexer(const qsfm_indexer_params* p, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * Norm of the queries and keys of each head with the position rotation in
 * the same pass, and the store of the key rows into the cache that the
 * attention reads. An addition of this library: the step that makes what
 * qsfm_forward() takes. For each query token t, each head row x of q (and
 * the token's one latent row of kv), of dim = 512 elements:
 *   y = x / sqrt(mean(x^2) + eps) * weight          (norm_q / norm_kv set;
 *                                                    else y = x)
 *   the rope_dim elements from rope_offset on are rotated by the angles of
 *   positions[t]: (a, b) -> (a cos - b sin, b cos + a sin) with the pairs
 *   (2i, 2i + 1) when interleaved is set, (i, i + rope_dim / 2) otherwise,
 *   cos = cos_sin[pos][i], sin = cos_sin[pos][rope_dim / 2 + i]
 * in fp32, rounded once: q_out[t] in bf16; the kv row, whose fp32 values are
 * carried with what they leave over so that every code is the formula's, in
 * the row format kv_layout at row slot_map[t] of the cache (kv_cache is
 * [num_blocks, 128, 1, row], row s its s-th row).
 *   packed384  exponent byte 127 + E, E = floor(log2 max|y|) - 10 over the
 *              whole row (clipped to -100 .. 100), scale = e4m3(max|y| of the
 *              16 / 6 / 2^E), code = e2m1(y / (scale 2^E)), to nearest even,
 *              saturating
 *   packed640  exponent of each 64 nope elements the smallest with max|y| <=
 *              448 2^(e - 127) (e clipped to 27 .. 227), code = e4m3(y / 2^(e - 127))
 *   fp8        scale = max|y| of each 64 / 448 (at least 1e-12 / 448), code =
 *              e4m3(y / scale), scale as it is before its rounding to fp32
 *              (the root that both share is fp32's: stored scales are within
 *              20 2^-24 of the formula's)
 *   A scale group with an element that is not finite stores a scale of NaN (fp8
 *   rows: and codes of NaN); the other groups are as without it. Elements that are
 *   stored as bf16 are stored as they are.
 * A token whose position is negative is padding: nothing is written for it. A
 * slot that is negative stores no row (q_out and kv_out are
 * written); each slot is named by at most one token (of two, the row's bytes
 * are a mixture). A position past the table skips the token
 * (QSFM_FAULT_POSITION), a slot past the cache the store (QSFM_FAULT_SLOT).
 *
 *   q          [T, heads, 512] bf16, fp16 or fp32 (in_type), element strides
 *              q_token_stride and q_head_stride, or NULL (heads = 0)
 *   kv         [T, 512] of the same type, kv_token_stride, or NULL
 *   q_out      bf16 [T, heads, 512] contiguous; may be q itself where q is
 *              bf16 and contiguous
 *   kv_cache   NULL: no row is stored; kv_scale fp32 [num_blocks, 128, 1, 8]
 *              for fp8 rows, else NULL
 *   kv_out     bf16 [T, 512] or NULL: the values of the stored rows (rounded
 *              to bf16 for fp8 rows, exact otherwise; without kv_cache the
 *              rows of format bf16)
 *   q_weight, kv_weight  [512] fp32, or bf16 (weights_bf16), or NULL (ones)
 *   positions  int32 [T]; cos_sin fp32 [max_positions, rope_dim], both NULL
 *              with rope_dim 0 (positions may be given all the same)
 *   slot_map   int32 [T], required with kv_cache
 * rope_dim is 0 or 32, 64, 128 or 256 and rope_offset a multiple of it.
 * Pointers and strides: q, kv, q_out, kv_cache, kv_out, the weights and
 * cos_sin 16-byte aligned, strides multiples of 16 bytes; the rest 4-byte.
 * Outputs overlap no input (QSFM_ERR_INVALID_ARG) but for q_out = q.
 */
typedef enum { QSFM_BF16 = 0, QSFM_F16 = 1, QSFM_F32 = 2 } qsfm_elem_type;

typedef struct qsfm_norm_rope_params {
  int32_t tokens;          /* T                                             */
  int32_t heads;           /* head rows of a token in q; 0 without q        */
  int32_t dim;             /* must be 512                                   */
  int32_t in_type;         /* qsfm_elem_type of q and kv                    */
  int32_t weights_bf16;    /* non-zero: q_weight and kv_weight are bf16     */
  int32_t norm_q;          /* non-zero (default): normalise the query rows  */
  int32_t norm_kv;         /* non-zero (default): normalise the kv rows     */
  int32_t rope_dim;
  int32_t rope_offset;
  int32_t interleaved;
  int32_t max_positions;   /* rows of cos_sin                               */
  int32_t kv_layout;       /* qsfm_kv_layout of kv_cache                    */
  int32_t num_blocks;      /* blocks of 128 rows in kv_cache                */
  float eps;
  int64_t q_token_stride, q_head_stride, kv_token_stride; /* in elements    */
  const void* q;
  const void* kv;
  const void* q_weight;
  const void* kv_weight;
  const float* cos_sin;
  const int32_t* positions;
  const int32_t* slot_map;
  void* q_out;
  void* kv_cache;
  float* kv_scale;
  void* kv_out;
} qsfm_norm_rope_params;

/* Defaults: dim 512, both norms, eps 1e-6, kv_layout fp8, pointers NULL. */
void qsfm_norm_rope_params_init(qsfm_norm_rope_params* p);

/* One launch on `stream` (none for T = 0, whose pointers are not looked at); no
 * workspace, nothing read back. Errors:
 * QSFM_ERR_INVALID_ARG, QSFM_ERR_UNSUPPORTED (dim other than 512, rope_dim
 * not built, T (heads + 1) above 2^30, a cache of 2^31 rows or more). */
qsfm_status qsfm_norm_rope_store(const qsfm_norm_rope_params* p, void* stream);

/*
 * Block tables and slots from request lengths, on the GPU. An addition of
 * this library: the bookkeeping of the paged cache between two steps. With
 * rows(n) = floor(n / cmp_ratio), held_b = ceil(rows(prev_lens[b]) / 128) and
 * need_b = ceil(rows(lens[b]) / 128), for the B requests in order:
 *   a request that shrinks gives the blocks of its table columns need_b ..
 *   held_b - 1 back to the end of the free list (a request that has ended has
 *   lens[b] = 0; a column of -1 holds no block and gives none back), then a
 *   request that grows takes the blocks of columns held_b .. need_b - 1 from the
 *   end of the list, in the order (request, column). So a block given back in a
 *   call may be taken in the same call.
 * The table columns behind need_b are left as they were.
 * The new rows rows(prev_lens[b]) .. rows(lens[b]) - 1 of all requests, end to
 * end, are described by
 *   slot_map   int32 [max_rows]  row of the pool: table[b][row / 128] * 128 +
 *              row % 128; -1 where no block was left and behind the last row
 *   positions  int32 [max_rows] or NULL: row * cmp_ratio; -1 behind the last
 *   cu_rows    int32 [B + 1] or NULL: the rows' prefix sums (with cmp_ratio 1
 *              the cu_seqlens_q of the step)
 *   residual   int32 [B] or NULL: lens[b] - rows(lens[b]) * cmp_ratio
 *              (cmp_residual_kv)
 * block_table int32 [B, max_blocks], free_list int32 [free_capacity] and
 * free_count int32 [1] are the state, updated in place; free_count_out, when
 * not NULL, takes the new count instead of free_count (the call can then be
 * repeated on the same inputs). Bad data is reported in the fault word and
 * skipped: no free block left (QSFM_FAULT_BLOCK_POOL: -1 in the table); a
 * block id outside [0, num_blocks) on the free list or in a held column that a
 * new row falls into, and one outside [-1, num_blocks) in a column given back
 * (QSFM_FAULT_ORI_BLOCK_ID: -1 in the table, slots -1, not given back); more
 * than max_blocks blocks in a request (QSFM_FAULT_ORI_TABLE_COL), more new
 * rows than max_rows (QSFM_FAULT_SLOT). Negative lengths count as 0. The
 * buffers do not overlap.
 */
typedef struct qsfm_block_table_params {
  int32_t batch;           /* B, at most 8192                               */
  int32_t max_blocks;      /* block_table row width                         */
  int32_t num_blocks;      /* blocks in the pool                            */
  int32_t free_capacity;   /* entries of free_list                          */
  int32_t max_rows;        /* entries of slot_map and positions             */
  int32_t cmp_ratio;       /* 1 .. 128                                      */
  int32_t block_size;      /* must be 128                                   */
  int32_t* block_table;
  const int32_t* prev_lens;
  const int32_t* lens;
  int32_t* free_list;
  int32_t* free_count;
  int32_t* free_count_out;
  int32_t* slot_map;
  int32_t* positions;
  int32_t* cu_rows;
  int32_t* residual;
} qsfm_block_table_params;

/* Defaults: cmp_ratio 1, block size 128, all pointers NULL. */
void qsfm_block_table_params_init(qsfm_block_table_params* p);

/* One launch on `stream`, two where max_rows is above 8192 and the count is
 * updated in place; no workspace, nothing read back. Errors:
 * QSFM_ERR_INVALID_ARG, QSFM_ERR_UNSUPPORTED (more than 8192 requests, a
 * block size other than 128, a pool of 2^31 rows or more, max_blocks * 128 or
 * max_rows or B * max_blocks above 2^30). */
qsfm_status qsfm_update_block_tables(const qsfm_block_table_params* p, void* stream);

/*
 * Rows quantised to e4m3 with an fp32 scale per 128 elements. An addition of
 * this library: the form that qsfm_lightning_indexer() takes queries and keys in
 * (a head of 128 elements has one scale) and qsfm_scaled_matmul() its rows.
 * Row t of the K = heads * dim elements y, with A = max|y| of each 128 elements
 * (the last scale of a row may have fewer):
 *   scale = A / 448 and code = e4m3(448 y / A), A at least 1e-12; with
 *   pow2_scale, scale = 2^e, e the smallest with A <= 448 2^e (clipped to -100 ..
 *   100), and code = e4m3(y / scale); to nearest even, saturating.
 *   y = x, silu(gate) * x when gate is given, or x with the rope_dim elements of
 *   each head row from rope_offset on turned by the angles of positions[t], as
 *   qsfm_norm_rope_store() turns them, or turned back when inverse is set (the
 *   attention's output, whose values carry the keys' rotation).
 * Every code is that of the formula (a gate below -87 counts as silu = 0). Turned
 * and gated y are taken to about 46 bits, those of its terms when turned: a quotient
 * nearer than that to the border of two codes may have either. Scales
 * that are not powers of two are the formula's rounded to fp32, or where A is a
 * computed y within a few units of 2^-24 of it: 4 when turned, 11 + 1.25 |gate|
 * when gated. A group with an element y that is not finite has codes and a
 * scale of NaN; so has one with a y, or a term of a turned y, above fp32's largest
 * number.
 *   x, gate    bf16, fp16 or fp32 (in_type) [source_rows, heads, dim], element
 *              strides *_row_stride and *_head_stride, elements contiguous
 *   row_index  int32 [T] or NULL: row t is made of row row_index[t] of x and gate
 *              (without it source_rows must be T)
 *   positions  int32 [T]; cos_sin fp32 [max_positions, rope_dim], both NULL with
 *              rope_dim 0 (positions may be given all the same)
 *   codes      e4m3fn bytes [T, K];  scale fp32 [T, ceil(K / 128)]
 * A row whose index or position is negative is padding: nothing is written for it.
 * A row whose index is past the source rows (QSFM_FAULT_ROW_INDEX) or whose position
 * is past the table (QSFM_FAULT_POSITION) is skipped.
 * K is a multiple of 16, dim of 128 with more than one head; rope_dim is 0, 32, 64
 * or 128 and rope_offset a multiple of it; gate and a rotation exclude each other.
 * x, gate, cos_sin, codes 16-byte aligned, strides multiples of 16 bytes, the rest
 * 4-byte aligned. Outputs overlap no input.
 */
typedef struct qsfm_quantize_params {
  int32_t rows;            /* T                                             */
  int32_t source_rows;     /* rows of x and gate                            */
  int32_t heads;           /* default 1                                     */
  int32_t dim;
  int32_t in_type;         /* qsfm_elem_type of x and gate                  */
  int32_t pow2_scale;
  int32_t rope_dim;
  int32_t rope_offset;
  int32_t interleaved;     /* pairs (2i, 2i + 1); else (i, i + rope_dim / 2) */
  int32_t inverse;
  int32_t max_positions;   /* rows of cos_sin                               */
  int64_t x_row_stride, x_head_stride, gate_row_stride, gate_head_stride; /* in elements */
  const void* x;
  const void* gate;
  const int32_t* row_index;
  const int32_t* positions;
  const float* cos_sin;
  void* codes;
  float* scale;
} qsfm_quantize_params;

/* Defaults: one head, pointers NULL. */
void qsfm_quantize_params_init(qsfm_quantize_params* p);

/* One launch on `stream`, two for many heads that are turned (none for T = 0, whose
 * pointers are not looked at); no workspace, nothing read back. Errors: QSFM_ERR_INVALID_ARG,
 * QSFM_ERR_UNSUPPORTED (K not a multiple of 16, heads of a dim that is not one of
 * 128, rope_dim not built, T ceil(K / 128) of 2^31 - 2^16 or more, a stride of 2^31 or more). */
qsfm_status qsfm_quantize_rows(const qsfm_quantize_params* p, void* stream);

/*
 * Product of quantised rows with quantised matrices. An addition of this library:
 * the projections around the attention, and the experts' products.
 *   out[m][j] = sum over blocks b of 128 of  a_scale[m][b] w_scale[g][j / 128][b]
 *                 * (sum over k in b of a[m][k] w[g][j][k])
 * with e4m3fn a and w; g is 0, or with cu_rows the group of row m, the g with
 * cu_rows[g] <= m < cu_rows[g + 1]. The two scales of a block are multiplied in fp32
 * (above its largest number their product is inf, below 2^-126 it has fewer bits), the sum
 * over a block is the tensor cores' (fp32 accumulators), blocks are added in fp32, and the
 * result is rounded once to out_type. A call gives the same bits every time; for
 * another number of rows the blocks may be added in another order.
 *   a          e4m3fn bytes [M, K], rows a_row_stride apart
 *   a_scale    fp32 [M, ceil(K / 128)], element strides a_scale_row_stride and
 *              a_scale_col_stride
 *   w          e4m3fn bytes [groups, N, K], strides w_group_stride, w_row_stride
 *   w_scale    fp32 [groups, ceil(N / 128), ceil(K / 128)]
 *   cu_rows    int32 [groups + 1] or NULL (one group, all rows): rows of group g;
 *              groups may be empty. Rows before the first and behind the last group
 *              are left as they were. Entries that decrease or lie outside 0 .. M are
 *              cut to what is there (QSFM_FAULT_GROUP_ROWS)
 *   out        [M, N] of out_type, rows out_row_stride apart (elements)
 * K is a multiple of 16. a, w: 16-byte aligned, strides multiples of 16 bytes; out
 * aligned to its elements, the rest 4-byte aligned. out overlaps no input.
 */
typedef struct qsfm_matmul_params {
  int32_t rows;            /* M                                             */
  int32_t n;
  int32_t k;
  int32_t groups;          /* default 1                                     */
  int32_t out_type;        /* qsfm_elem_type                                */
  int64_t a_row_stride, w_row_stride, w_group_stride;
  int64_t a_scale_row_stride, a_scale_col_stride;
  int64_t out_row_stride;
  const void* a;
  const float* a_scale;
  const void* w;
  const float* w_scale;
  const int32_t* cu_rows;
  void* out;
} qsfm_matmul_params;

/* Defaults: one group, bf16 output, pointers NULL. */
void qsfm_matmul_params_init(qsfm_matmul_params* p);

/* One launch on `stream` (none for M = 0, whose pointers are not looked at); no
 * workspace, nothing read back. Errors: QSFM_ERR_INVALID_ARG,
 * QSFM_ERR_UNSUPPORTED (K not a multiple of 16, more than 1024 groups, M, N or K of
 * 2^24 or more, more than 2^30 tiles of 128 x 128 outputs, a stride of 2^36 or more). */
qsfm_status qsfm_scaled_matmul(const qsfm_matmul_params* p, void* stream);

/* How qsfm_scaled_matmul() would compute this product on the current device, for
 * tests: the rows and columns of out that a tile has, and the parts that a tile's
 * blocks of K are split into. Launches nothing. QSFM_ERR_INVALID_ARG for M = 0 or a
 * NULL output. */
qsfm_status qsfm_debug_matmul_plan(const qsfm_matmul_params* p, int32_t* tile_rows, int32_t* tile_columns,
                                   int32_t* parts);

/* Synchronously read and clear the device fault word of the current
 * device (QSFM_FAULT_* bits). Returns QSFM_ERR_DEVICE_FAULT when non-zero. */
qsfm_status qsfm_get_device_status(int32_t* fault_word);

const char* qsfm_status_string(qsfm_status s);
int32_t qsfm_abi_version(void);

/* The CUDA runtime error code behind the last QSFM_ERR_CUDA an entry point
 * returned on the calling host thread (0 if none), and its name in *name
 * when name is not NULL (a static string). Not cleared by later calls. */
int32_t qsfm_last_cuda_error(const char** name);

#ifdef __cplusplus
}
#endif

#endif /* QSFM_H */
