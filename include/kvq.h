/*
 * kvq.h -- C ABI of libkvq: quantize-on-write into a paged KV cache and paged
 * decode attention that reads the packed low-bit cache and folds
 * dequantization into its load path.  One process, one NVIDIA GB300 GPU
 * (sm_103a).
 *
 * Sources of the operations (web pages, by title and section):
 *  [P1] "KV Cache 量化深度解析：Per-Tensor、Per-Token-Head 与 NVFP4":
 *       sec. 二 (the KVQuantMode enum: NONE, FP8_PER_TENSOR, INT8/FP8
 *       PER_TOKEN_HEAD, NVFP4), sec. 2.1, 2.2, 2.3.
 *  [P2] "KVarN：华为推出的原生 vLLM KV-cache 量化后端，打破性能与精度的权衡":
 *       技术原理 (tile, Hadamard rotation, variance normalisation, asymmetric
 *       RTN), 配置与部署 (preset kvarn_k4v2_g128), 注意事项 (tile = page = 128).
 *  [P3] "KV Cache 量化 · LLM Glossary": s = max|x|/127, q = clip(round(x/s)),
 *       dequantize while loading inside the attention kernel.
 *  [P4] "KV 量化" (rustineverything.app): 写和读 (the write call takes the
 *       cache dtype and the k/v scales, the read multiplies by the descale;
 *       FP8 stored as uint8 bit patterns), per-token-head and NVFP4 scales
 *       stored inside the page next to the data.
 *  [P5] "NVFP4 KV Cache：Blackwell 上的 4-bit 缓存量化": two-level scaling,
 *       KV write/read paths, attention A = softmax(QK^T/sqrt(d)), O = AV;
 *       an unsupported combination is an immediate error, not a silent
 *       fallback; "用一组数直观看缩放的作用" (the nvfp4_4over6 mode picks a
 *       max/6 or max/4 block scale by reconstruction error).
 *  [P4] also names int4_per_token_head: head_size/2 bytes of data plus one
 *       fp32 scale per token and kv head.
 *
 * Conventions
 *  - Every call returns a kvq_status; KVQ_OK is 0.  On error,
 *    kvq_last_error() returns a message (thread-local, valid until the next
 *    call on the same thread).  Argument errors are detected on the host
 *    before anything is launched.
 *  - Pointers named dev_* or documented as device pointers are CUDA device
 *    memory owned by the caller.  The library never allocates device memory:
 *    the cache pool and the decode workspace are caller buffers (the one
 *    library-owned buffer is the fixed scratch array described at
 *    kvq_decode_attention_noalloc).  A kvq_cache handle owns only a small
 *    host-side descriptor.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  All device
 *    work is enqueued on it asynchronously, unless a call says otherwise.
 *  - There is no fallback path: an unsupported combination of mode, head_dim,
 *    page_size or dtype returns KVQ_ERR_UNSUPPORTED.
 *  - Errors that only the device can see (a slot or page id out of range, a
 *    KVarN write that is not whole tiles, a seq_len above its bound) never
 *    fault: the offending token or tile is skipped and a bit is set in the
 *    cache's device error word; kvq_cache_read_errors() fetches it.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int kvq_status;
#define KVQ_OK 0
#define KVQ_ERR_INVALID_ARG 1   /* null pointer, negative size, misaligned buffer, ... */
#define KVQ_ERR_UNSUPPORTED 2   /* mode / head_dim / page_size / dtype combination */
#define KVQ_ERR_MODE_MISMATCH 3 /* call mode differs from the cache's mode */
#define KVQ_ERR_CAPACITY 4      /* buffer too small for the layout or the plan */
#define KVQ_ERR_CUDA 5          /* a CUDA runtime/driver call failed */
#define KVQ_ERR_DEVICE_CHECK 6  /* the device error word is non-zero */

/* Quantization modes ([P1] sec. 二 enum values, plus the KVarN preset of [P2]). */
typedef enum {
  KVQ_FP8_PER_TENSOR = 1,      /* E4M3 payload, one fp32 scale per side (K, V) */
  KVQ_INT8_PER_TOKEN_HEAD = 2, /* int8 payload, fp32 scale per token x kv head, s = max|x|/127 */
  KVQ_FP8_PER_TOKEN_HEAD = 3,  /* E4M3 payload, fp32 scale per token x kv head, s = max|x|/448 */
  KVQ_NVFP4 = 4,               /* E2M1 payload, E4M3 scale per 16 values, fp32 global scale */
  KVQ_INT4_PER_TOKEN_HEAD = 5, /* signed 4-bit payload, fp32 scale per token x kv head, s = max|x|/7 */
  KVQ_NVFP4_4OVER6 = 6,        /* NVFP4 storage; each block scale is max/6 or max/4, by error */
  KVQ_KVARN_K4V2_G128 = 16     /* 4-bit keys, 2-bit values, 128-token tiles */
} kvq_mode;

typedef enum { KVQ_F16 = 0, KVQ_F32 = 1 } kvq_dtype;

/* Device error bits (kvq_cache_read_errors). */
#define KVQ_DEVERR_SLOT_RANGE 0x1u   /* a write slot >= num_pages * page_size */
#define KVQ_DEVERR_PAGE_RANGE 0x2u   /* a block_table entry outside [0, num_pages) */
#define KVQ_DEVERR_PARTIAL_TILE 0x4u /* KVarN: a write or a sequence that is not whole tiles, or an
                                        append carrying rows of two tiles of one sequence */
#define KVQ_DEVERR_SEQ_LEN 0x8u      /* a seq_len above max_seq_len or max_pages * page_size */
#define KVQ_DEVERR_TIMEOUT 0x10u     /* a bounded wait on a copy ran out (work skipped) */
#define KVQ_DEVERR_SEQ_ID 0x20u      /* kvq_kvarn_append: a seq_id outside [0, num_seqs) */
#define KVQ_DEVERR_POSITION 0x80u    /* kvq_norm_rope_write, kvq_latent_write: a position outside [0, max_position) */
#define KVQ_DEVERR_QUERY_RANGE 0x100u /* kvq_chunk_attention and the latent calls: cu_q_lens (or cu_k_lens) of a
                                        sequence not an ascending range of at most max_q_len rows of the batch */
#define KVQ_DEVERR_BOUNDS 0x40u      /* debug build only: a store fell outside the buffer its
                                        arguments describe (skipped); see kvq_debug_build */

typedef struct {
  int32_t num_pages;    /* pages in the pool */
  int32_t page_size;    /* tokens per page: 16 (modes 1-4) or 128 (KVarN) */
  int32_t num_kv_heads; /* Hkv */
  int32_t head_dim;     /* D: 32 or 128 (modes 1-4), 128 (KVarN) */
  int32_t mode;         /* kvq_mode */
  int32_t io_dtype;     /* kvq_dtype of the K/V written and of the decode query */
} kvq_cache_config;

typedef struct kvq_cache kvq_cache;

/* Pool layout (little-endian, version 1).  The pool is a 256-byte header
 * followed by one block per (page, kv head), page-major:
 *   block(p, h) at byte 256 + (p * num_kv_heads + h) * block_bytes.
 * Token t of page p is row t of that block.  Per mode (P = page_size, D = head_dim):
 *   FP8 per-tensor : K[P][D] e4m3 | V[P][D] e4m3                    (2PD bytes)
 *   INT8 / FP8 PTH : K[P][D] | V[P][D] | K scale[P] f32 | V scale[P] f32
 *   NVFP4, 4over6  : K[P][D/2] | V[P/2][D] | K s_b[P][D/16] e4m3 | V s_b[P][D/16] e4m3
 *   INT4 PTH       : K[P][D/2] | V[P/2][D] | K scale[P] f32 | V scale[P] f32
 *   KVarN (P=D=128): K[128][64] u4 | V[128][32] u2 |
 *                    K scale[D] zero[D] c[D] r[P] f32 | V scale[P] zero[P] r[P] c[D] f32
 * 4-bit codes: NVFP4 K (E2M1) the even head_dim index in the low nibble;
 * NVFP4 V byte [k][d] holds channel d of tokens 2k (low nibble) and 2k+1 --
 * the pairing decode's tensor-core fragments take, with no nibble shuffling.
 * INT4 (two's complement) in 32-bit little-endian words, nibble k = bits
 * 4k..4k+3: a K row word m holds channel 8m + 2k in nibble k < 4 and
 * 8m + 2(k-4) + 1 in nibble k >= 4; a V pair row [k] word m holds channel
 * 4m + k of token 2k' = 2k in nibble k < 4 and channel 4m + k - 4 of token
 * 2k + 1 in nibble k >= 4 -- the orders one lop3 turns into f16 pairs.
 * 2-bit codes: element 4i+j in bits 2j..2j+1 of byte i.  The header holds, at byte 16 and
 * 20, the per-tensor K and V scales (FP8 per-tensor s; NVFP4 s_t), and at
 * byte 12 the device error word.  This is the same content as the in-page
 * layouts of [P4] (data plus one fp32 scale per token-head; head_size/2 bytes
 * of FP4 then head_size/16 bytes of E4M3 block scales), with each kind of
 * field gathered into its own 16-byte-aligned sub-array. */

const char* kvq_last_error(void);
int kvq_version(void); /* layout/ABI version, currently 1 */

/* 1 when the library was built with -DKVQ_DEBUG=1, else 0.  In such a build
 * every global store of every kernel first checks that its bytes lie inside
 * the buffer its arguments describe (the pool, the tail buffer, the output,
 * the workspace); a store that does not is skipped and KVQ_DEVERR_BOUNDS is
 * set in the cache's error word.  It stands in for a memory checker: an
 * indexing fault shows up as a flag instead of a corrupted neighbour.  A
 * release build checks nothing and never sets KVQ_DEVERR_BOUNDS. */
int kvq_debug_build(void);

/* Debug builds only (KVQ_ERR_UNSUPPORTED otherwise): one kernel tries a store
 * one byte past the end of the pool's header span, which lies inside the
 * pool's memory, and so must set KVQ_DEVERR_BOUNDS and leave the byte as it
 * was.  Lets a test see that the checks are live.  Enqueued on `stream`. */
kvq_status kvq_debug_bounds_selftest(kvq_cache* cache, void* stream);

/* Bytes of the pool for `cfg` (header included), and of one (page, kv head)
 * block.  No device work. */
kvq_status kvq_cache_bytes(const kvq_cache_config* cfg, size_t* bytes);
kvq_status kvq_cache_block_bytes(const kvq_cache_config* cfg, size_t* bytes);

/* Bind a cache descriptor to the caller's device buffer `dev_buf` (at least
 * kvq_cache_bytes bytes, 256-byte aligned).  Writes the header (scales = 1.0,
 * error word = 0) synchronously; page contents are left as they are.
 * `*out` is freed with kvq_cache_free, which never touches device memory. */
kvq_status kvq_cache_alloc(const kvq_cache_config* cfg, void* dev_buf, size_t bytes, kvq_cache** out);
kvq_status kvq_cache_free(kvq_cache* cache);

/* Per-tensor scales ([P1] sec. 2.1 K_fp8 = K/scale; [P5] s_t), written into
 * the header on `stream`.  Used by KVQ_FP8_PER_TENSOR (s) and the two NVFP4
 * modes (s_t); other modes ignore them.  Scales must be finite and > 0. */
kvq_status kvq_cache_set_tensor_scales(kvq_cache* cache, float k_scale, float v_scale, void* stream);

/* amax = max |x| over n elements of `x` (device, dtype kvq_dtype), written
 * to the device float *dev_out (overwritten, not accumulated).  Exact. */
kvq_status kvq_tensor_amax(const void* x, int dtype, size_t n, float* dev_out, void* stream);

/* Set the header's scales from device amax values without a host round trip:
 * FP8 per-tensor s = amax/448, NVFP4 (both modes) s_t = amax/(448*6); an amax of 0 gives
 * 1.0.  Both pointers are device floats (e.g. from kvq_tensor_amax). */
kvq_status kvq_cache_set_tensor_scales_from_amax(kvq_cache* cache, const float* dev_amax_k,
                                                 const float* dev_amax_v, void* stream);

/* Copy the device error word to *flags (synchronises `stream`); if `clear`,
 * reset it to 0 afterwards. */
kvq_status kvq_cache_read_errors(kvq_cache* cache, uint32_t* flags, int clear, void* stream);

/* Quantize-on-write ([P4] 写和读; [P1] sec. 2.1-2.3; [P2] 技术原理).
 *  k, v          device [num_tokens][num_kv_heads][head_dim], io_dtype of the cache
 *  slot_mapping  device int32 [num_tokens]: slot = page * page_size + row;
 *                a negative slot skips the token; a slot past the pool skips it
 *                and sets KVQ_DEVERR_SLOT_RANGE.
 *  mode          must equal the cache's mode (else KVQ_ERR_MODE_MISMATCH).
 * Per mode: FP8 per-tensor q = E4M3(x/s) with the header scale; INT8/FP8
 * per-token-head s = max(max|x|, 1e-8)/127 (or /448), q = clip(rint(x/s)) (or
 * E4M3(x/s)); INT4 per-token-head s = max(max|x|, 1e-8)/7, q = clip(rint(x/s),
 * -7, 7); NVFP4 s_b = E4M3(max_block|x| / (6 s_t)), q = E2M1(x/(s_t s_b));
 * NVFP4 4over6: the same block coded with s_b = E4M3(max_block|x| / (4 s_t))
 * as well, keeping the coding whose fp32 sum of squared reconstruction errors
 * (x - s_t s_b q)^2, summed as a pairwise tree of neighbours, is smaller
 * (max/6 on a tie);
 * KVarN: num_tokens must be a multiple of 128 and every 128 consecutive tokens
 * must fill one page in order (slot_mapping[128i + j] = 128 page + j); a tile
 * that does not is skipped with KVQ_DEVERR_PARTIAL_TILE.  All divisions are
 * IEEE round-to-nearest; results are bit-identical to the specification. */
kvq_status kvq_quantize_write(kvq_cache* cache, const void* k, const void* v,
                              const int32_t* slot_mapping, int num_tokens, int mode, void* stream);

/* ---- Reading back --------------------------------------------------------
 * The values the cache holds at `slot_mapping`, as dense rows: codes times
 * their scales in fp32 (NVFP4 code s_b s_t), rounded once to out_dtype; KVarN
 * rows r_t c_d (scale q + zero) rotated back to the input domain by the
 * normalised Hadamard transform in fp32.  ([P3]: x^ = q s; [P5] KV 的写入与读取路径.)
 *  slot_mapping  device int32 [num_tokens]; a negative slot leaves its output
 *                rows as they were; a slot past the pool does too and sets
 *                KVQ_DEVERR_SLOT_RANGE.  The same slot may appear twice.
 *  k_out, v_out  device [num_tokens][num_kv_heads][head_dim], out_dtype,
 *                16-byte aligned; either may be NULL (that side is not read)
 * KVarN reads quantized tiles only (an open tile's rows are in the caller's
 * tail buffer as they were written).  A value outside the fp16 range reads as
 * infinity at out_dtype KVQ_F16. */
kvq_status kvq_cache_read(const kvq_cache* cache, const int32_t* slot_mapping, int num_tokens, void* k_out,
                          void* v_out, int out_dtype, void* stream);

/* ---- Norm, rotation and quantized write in one pass -----------------------
 * For every token and head, with x the head's row of head_dim values:
 *   y = x w / sqrt(mean(x^2) + eps)              (y = x where the weight is NULL)
 *   the first rot_dim values of y are rotated by the token's angles: for pair i
 *   of rot_dim / 2, (a, b) = values (i, i + rot_dim/2), or (2i, 2i + 1) when
 *   `interleaved`:  a' = a cos_i - b sin_i,  b' = b cos_i + a sin_i
 * and the result is rounded once to io_dtype.  Queries go to q_out; keys (from
 * their rounded rows) and values are quantized into the cache as by
 * kvq_quantize_write, whose rules for slots hold here too: the slots of one
 * call are distinct, a negative slot writes nothing to the cache, a slot past
 * the pool sets KVQ_DEVERR_SLOT_RANGE.  The rotated rows are the correctly
 * rounded values of the formula (evaluated to about 2^-44 where fp32 does not
 * settle the rounding; fp32 results below 2^-90 only to 2^-22).  Infinities and
 * NaN follow the formula by IEEE rules; values past rot_dim meet no others.
 * All pointers are device pointers, 16-byte aligned (positions, slot_mapping: 4). */
typedef struct {
  const void* q;      /* io_dtype, token t's heads at q + t * q_stride: [num_q_heads][head_dim] */
  const void* k;      /* [num_kv_heads][head_dim] at k + t * k_stride */
  const void* v;      /* likewise; may be NULL without slot_mapping */
  int64_t q_stride;   /* elements between tokens (a fused projection's row); multiples of 16 bytes */
  int64_t k_stride;
  int64_t v_stride;
  const int32_t* positions;  /* [num_tokens]; one outside [0, max_position) skips its token (its q_out and
                                k_out rows stay as they were) and sets KVQ_DEVERR_POSITION */
  const float* cos_sin;      /* [max_position][rot_dim]: rot_dim/2 cosines, then rot_dim/2 sines */
  const void* q_weight;      /* [head_dim] io_dtype, or NULL: no norm of the queries */
  const void* k_weight;      /* [head_dim] io_dtype, or NULL: no norm of the keys */
  const int32_t* slot_mapping; /* [num_tokens], or NULL: the cache is not written */
  void* q_out;        /* [num_tokens][num_q_heads][head_dim], io_dtype; may be q itself where q is dense */
  void* k_out;        /* [num_tokens][num_kv_heads][head_dim] rotated keys, or NULL; may be k itself */
  int32_t num_tokens;
  int32_t num_q_heads;
  int32_t rot_dim;      /* a multiple of 16, at most head_dim; 0 rotates nothing (positions and cos_sin
                           are not read and may be NULL) */
  int32_t max_position; /* rows of cos_sin */
  int32_t interleaved;
  float eps;            /* >= 0 */
} kvq_norm_rope;
/* KVarN quantizes whole tiles: there slot_mapping must be NULL, and k_out and v
 * go to kvq_kvarn_append or kvq_quantize_write (else KVQ_ERR_UNSUPPORTED). */
kvq_status kvq_norm_rope_write(kvq_cache* cache, const kvq_norm_rope* r, int mode, void* stream);

/* Decode plan: how many KV splits per (sequence, kv head), the tokens per
 * split, and the workspace bytes kvq_decode_attention needs for these sizes
 * (0 when a single split suffices, and 0 when the splits of each query row
 * merge on chip: 2 to 8 splits of the one-query kernel whose CTAs are all
 * resident at once run as one thread-block cluster per row, so that no split
 * partial goes through memory and no combine kernel is launched).
 * max_seq_len is a host-side upper bound of every seq_len. */
kvq_status kvq_decode_plan(const kvq_cache* cache, int num_seqs, int num_q_heads, int max_seq_len,
                           int* num_splits, int* tokens_per_split, size_t* workspace_bytes);
kvq_status kvq_decode_workspace_bytes(const kvq_cache* cache, int num_seqs, int num_q_heads,
                                      int max_seq_len, size_t* bytes);

/* Paged decode attention over the packed cache ([P5] "K 与 V 的量化误差..."
 * A = softmax(QK^T/sqrt(d)), O = AV, one query per sequence; [P3]/[P5]:
 * dequantization happens in the kernel's load path, no dequantized copy of
 * the cache is made).
 *  q            device [num_seqs][num_q_heads][head_dim], io_dtype of the cache
 *  block_table  device int32 [num_seqs][max_pages]: page ids of each sequence
 *  seq_lens     device int32 [num_seqs]; 0 gives a zero output row
 *  max_seq_len  host upper bound of seq_lens (<= max_pages * page_size)
 *  softmax_scale  usually 1/sqrt(head_dim)
 *  out          device [num_seqs][num_q_heads][head_dim], dtype out_dtype
 *  workspace    device scratch of >= the planned bytes (may be NULL if 0)
 * GQA: query head h reads kv head h / (num_q_heads / num_kv_heads), which
 * must divide evenly with a group of at most 8.  KVarN: every seq_len must be
 * a multiple of 128 (whole tiles), the query is rotated by the same
 * normalised Hadamard transform and the output rotated back.
 * INT8, FP8 and INT4 per token and head: a weight times its value's scale is
 * held in steps of 2^-24 (fp32 io; 2^-26, 2^-28 and 2^-22 with fp16 io) and up to
 * 65504, so values far below 1 lose bits of their weights and fp32 values whose
 * scale passes 65504 become infinite.  The single tokens of kvq_chunk_attention are
 * held relative to their values' scales instead. */
kvq_status kvq_decode_attention(const kvq_cache* cache, const void* q, const int32_t* block_table,
                                int max_pages, const int32_t* seq_lens, int num_seqs,
                                int num_q_heads, int max_seq_len, int mode, float softmax_scale,
                                void* out, int out_dtype, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Multi-query decode: num_queries queries per sequence, as in speculative
 * decoding or a short prefill chunk, over the same packed pages ([P5] "K 与 V
 * 的量化误差进入 attention 的位置不同": A = softmax(QK^T/sqrt(d) + M), O = AV,
 * with M the causal mask).  q and out are [num_seqs][num_queries][num_q_heads]
 * [head_dim]; query i of sequence b stands at position seq_len_b - num_queries
 * + i and attends to tokens 0 .. seq_len_b - num_queries + i (none, output 0,
 * when that is negative).  Other arguments and rules are those of
 * kvq_decode_attention; num_seqs * num_queries <= 65535.  KVQ_KVARN_K4V2_G128
 * reads whole tiles only (every seq_len a multiple of 128, no open tile); a
 * query's causal prefix may end inside the last tile, whose later tokens it
 * does not see.  NVFP4 (and 4over6) and INT4 at head_dim 128 with
 * group * num_queries <= 64 read each page once for all the sequence's
 * queries (tensor-core columns = queries x heads); the other modes run each
 * query as one row of the decode grid over its causal prefix, the rows of a
 * sequence side by side so that the pages they share are mostly served from
 * L2.  Plan and workspace: kvq_decode_multi_plan /
 * kvq_decode_multi_workspace_bytes. */
kvq_status kvq_decode_multi_plan(const kvq_cache* cache, int num_seqs, int num_queries, int num_q_heads,
                                 int max_seq_len, int* num_splits, int* tokens_per_split, size_t* workspace_bytes);
kvq_status kvq_decode_multi_workspace_bytes(const kvq_cache* cache, int num_seqs, int num_queries,
                                            int num_q_heads, int max_seq_len, size_t* bytes);
kvq_status kvq_decode_attention_multi(const kvq_cache* cache, const void* q, const int32_t* block_table,
                                      int max_pages, const int32_t* seq_lens, int num_seqs, int num_queries,
                                      int num_q_heads, int max_seq_len, int mode, float softmax_scale,
                                      void* out, int out_dtype, void* workspace, size_t workspace_bytes,
                                      void* stream);

/* ---- Chunk attention -------------------------------------------------------
 * A batch of chunks of new tokens, of any lengths, over the paged cache that
 * already holds those tokens: prompts from their first token, chunks of long
 * prompts, drafted tokens, and single tokens, in one call ([P5] "K 与 V 的量化误差
 * 进入 attention 的位置不同": A = softmax(QK^T/sqrt(d) + M), O = AV; chunked
 * prefill and speculative decoding, 使用前仍应确认).  Query i of a sequence's m
 * queries stands at position p = seq_len - m + i; with s_t = softmax_scale q.k_t,
 *   logit_cap > 0:  s_t = logit_cap tanh(s_t / logit_cap)
 *   alibi_slopes:   s_t = s_t - alibi_slopes[head] |p - t|
 * it attends to the tokens t <= p, with window > 0 only those t > p - window,
 * and (with prefix_lens) all tokens t < prefix_len, before or after it, inside
 * the sequence.  A query at a negative position attends to nothing: output 0. */
typedef struct {
  float logit_cap;             /* 0: none; else 1e-10 to 1024, and at least softmax_scale / 1e30 */
  int32_t window;              /* 0: none */
  const float* alibi_slopes;   /* device [num_q_heads], or NULL */
  const int32_t* prefix_lens;  /* device [num_seqs], or NULL */
} kvq_attention_options;

/* Plan of a chunk attention: the parts a sequence's token range is split into
 * (for outputs of the cache's io_dtype), and the workspace bytes the call needs for
 * these sizes with either output type (0 where neither has more than one part).
 * max_q_len and max_seq_len are host upper bounds of the chunks and of
 * seq_lens; of `options` (NULL: none) only window and whether prefix_lens is
 * given matter.  Fewer rows may be split into more parts and need more bytes: a
 * workspace for batches of several sizes is the largest of their plans. */
kvq_status kvq_chunk_plan(const kvq_cache* cache, int total_q, int num_seqs, int num_q_heads, int max_q_len,
                          int max_seq_len, const kvq_attention_options* options, int* num_splits,
                          size_t* workspace_bytes);

/*  q            device [total_q][num_q_heads][head_dim], io_dtype of the cache
 *  cu_q_lens    device int32 [num_seqs + 1]: sequence b's queries are rows
 *               cu_q_lens[b] .. cu_q_lens[b+1] - 1 (a chunk may be empty; rows of
 *               no sequence are neither read nor written).  A sequence whose
 *               entries are not an ascending range of at most max_q_len rows
 *               inside [0, total_q] is skipped and sets KVQ_DEVERR_QUERY_RANGE.
 *  out          device [total_q][num_q_heads][head_dim], dtype out_dtype
 *  options      NULL: none
 * block_table, max_pages, seq_lens, max_seq_len, mode, softmax_scale and the
 * workspace are as for kvq_decode_attention, as is the rule for the head group.
 * A sequence's pages hold its queries' own tokens too (write them first).
 * Pages that lie wholly below every window (and past the prefix) are not read,
 * and their block_table entries not looked at.  Calls that may overlap on the
 * GPU need a workspace each.
 * Weights meet the values as pairs of fp16 numbers (2^-22 of a weight), held
 * relative to the largest weight times value scale that the row sees, whatever the
 * magnitudes.  (The value scales of one sequence may be 2^100 apart.)  Sums over
 * tokens are fp32: fp32 outputs are within 2e-5 of the sum of |weight x value|, about
 * 1e-6 as a rule; fp16 outputs at head_dim 128 within their rounding and 2^-27 for
 * each token of a part.
 * KVarN is not supported (KVQ_ERR_UNSUPPORTED): its open tile lies outside the
 * pages.  A token whose stored value codes or scale are not finite may make every
 * output of its sequence's chunk NaN, those of queries before it too. */
kvq_status kvq_chunk_attention(const kvq_cache* cache, const void* q, int total_q, const int32_t* cu_q_lens,
                               const int32_t* block_table, int max_pages, const int32_t* seq_lens, int num_seqs,
                               int num_q_heads, int max_q_len, int max_seq_len, int mode, float softmax_scale,
                               const kvq_attention_options* options, void* out, int out_dtype, void* workspace,
                               size_t workspace_bytes, void* stream);

/* ---- Latent caches ---------------------------------------------------------
 * A cache of one latent vector c_t (latent_dim values) and one rotated key part
 * r_t (rope_dim values) per token, shared by all query heads: with head h's
 * up-projections U_h (keys) and W_h (values), k_th = [U_h c_t, r_t] and
 * v_th = W_h c_t.  Attention reads it in either of two forms:
 *   absorbed   q' = [U_h^T q_h, q_rope]; scores q' . [c_t, r_t], outputs sum p_t c_t,
 *              which W_h takes to the head's values: kvq_latent_attention, over the
 *              paged latents, keys and values at once;
 *   expanded   the heads' own keys and values: kvq_latent_prompt_attention, over dense
 *              rows (kvq_latent_read gives the latents that a context has cached).
 * The latents are quantized as a row of kvq_quantize_write is, one scale per token
 * (or per tensor, or per 16 values); the rotary part is held in fp16.
 *
 * Pool layout: the 256-byte header, then one block per page of 16 tokens:
 *   FP8 per-tensor  : codes[16][L] e4m3 | rope[16][R] f16
 *   INT8 / FP8 PTH  : codes[16][L]      | rope[16][R] f16 | scale[16] f32
 *   NVFP4, 4over6   : codes[16][L/2]    | rope[16][R] f16 | s_b[16][L/16] e4m3
 * NVFP4 codes: the even index in the low nibble.  The header is that of the other
 * pools, the tensor scale at byte 16, the device error word at byte 12. */
typedef struct {
  int32_t num_pages;
  int32_t page_size;  /* 16 */
  int32_t latent_dim; /* L: 256 or 512 */
  int32_t rope_dim;   /* R: 64 */
  int32_t mode;       /* kvq_mode: FP8 per-tensor, INT8 or FP8 per-token(-head), NVFP4, NVFP4 4over6 */
  int32_t io_dtype;   /* kvq_dtype of the rows written and of the queries */
} kvq_latent_config;

typedef struct kvq_latent kvq_latent;

/* As kvq_cache_bytes, kvq_cache_alloc, kvq_cache_free and kvq_cache_read_errors; the
 * conventions on pointers, streams and errors are the same.  The handle is of its own
 * type: the calls above do not take it. */
kvq_status kvq_latent_bytes(const kvq_latent_config* cfg, size_t* bytes);
kvq_status kvq_latent_alloc(const kvq_latent_config* cfg, void* dev_buf, size_t bytes, kvq_latent** out);
kvq_status kvq_latent_free(kvq_latent* cache);
kvq_status kvq_latent_read_errors(kvq_latent* cache, uint32_t* flags, int clear, void* stream);

/* The per-tensor scale of FP8 per-tensor (s) and the NVFP4 modes (s_t), on `stream`: a
 * host value (finite, > 0), or from a device amax (kvq_tensor_amax): amax/448, amax/2688,
 * 1 for 0. */
kvq_status kvq_latent_set_scale(kvq_latent* cache, float scale, void* stream);
kvq_status kvq_latent_set_scale_from_amax(kvq_latent* cache, const float* dev_amax, void* stream);

/* Norm, rotation and quantized write of new tokens in one pass.  For token i
 *   c = x w / sqrt(mean(x^2) + eps)   (c = x where latent_weight is NULL)
 * and the rotary parts of its key and of its queries' heads are rotated by the table
 * row of its position, in half-split or interleaved pairs, as by kvq_norm_rope_write
 * with rot_dim = rope_dim.  Every result is the correctly rounded value in io_dtype;
 * the latent codes are those of that rounded row, and the key part is rounded from
 * there to fp16 (io_dtype fp32; beyond 65504 it becomes infinite).
 * The slots of one call are distinct; a negative slot writes nothing to the cache, one
 * past the pool sets KVQ_DEVERR_SLOT_RANGE; a position outside [0, max_position) skips its
 * token (all of its rows stay as they were) and sets KVQ_DEVERR_POSITION.  Rows and strides
 * are multiples of 16 bytes, in elements of io_dtype.  An output may be its own input. */
typedef struct {
  const void* latent;        /* [latent_dim] of token i at latent + i * latent_stride */
  const void* k_rope;        /* [rope_dim] at k_rope + i * k_rope_stride */
  const void* q_rope;        /* [rope_dim] of head h at q_rope + i * q_stride + h * q_head_stride, or NULL */
  void* q_rope_out;          /* likewise, by q_out_stride and q_out_head_stride: e.g. the tails of the absorbed
                                queries' rows; with q_rope only */
  int64_t latent_stride;
  int64_t k_rope_stride;
  int64_t q_stride, q_head_stride;
  int64_t q_out_stride, q_out_head_stride;
  const void* latent_weight; /* [latent_dim] io_dtype, or NULL: no norm */
  const int32_t* positions;  /* [num_tokens] */
  const float* cos_sin;      /* [max_position][rope_dim]: rope_dim/2 cosines, then rope_dim/2 sines */
  const int32_t* slot_mapping; /* [num_tokens], or NULL: the cache is not written */
  void* latent_out;          /* [num_tokens][latent_dim] io_dtype, dense, or NULL */
  void* k_rope_out;          /* [num_tokens][rope_dim] io_dtype, dense, or NULL */
  int32_t num_tokens;
  int32_t num_q_heads;       /* of q_rope */
  int32_t max_position;
  int32_t interleaved;
  float eps;                 /* >= 0 */
} kvq_latent_rows;
kvq_status kvq_latent_write(kvq_latent* cache, const kvq_latent_rows* r, int mode, void* stream);

/* The values the cache holds at `slot_mapping`, as by kvq_cache_read: latent_out
 * [num_tokens][latent_dim] and rope_out [num_tokens][rope_dim] in out_dtype; either may
 * be NULL. */
kvq_status kvq_latent_read(const kvq_latent* cache, const int32_t* slot_mapping, int num_tokens, void* latent_out,
                           void* rope_out, int out_dtype, void* stream);

/* Absorbed attention of ragged chunks of queries (a chunk of one is a decode step) over
 * the paged latents, which already hold the chunks' own tokens.  Query i of a
 * sequence's m stands at position seq_len - m + i and attends to the tokens up to it, or,
 * with causal = 0, to all of the sequence's tokens:
 *   s_t = softmax_scale (q[0..L) . c_t + q[L..L+R) . r_t),  out = sum softmax(s)_t c_t
 *  q            device [total_q][num_q_heads][latent_dim + rope_dim], io_dtype
 *  cu_q_lens    device int32 [num_seqs + 1], as for kvq_chunk_attention
 *  block_table  device int32 [num_seqs][max_pages]
 *  seq_lens     device int32 [num_seqs], at most max_seq_len <= max_pages * 16
 *  out          device [total_q][num_q_heads][latent_dim], out_dtype
 *  lse          device fp32 [total_q][num_q_heads]: log(sum exp(s_t)), or NULL
 * A query that sees no token: out 0, lse -infinity.  Rows of no sequence are neither
 * read nor written.  A page id outside the pool drops its tokens (KVQ_DEVERR_PAGE_RANGE).
 * A plan's num_splits is the most parts that a sequence's token range may be split into
 * (for outputs of io_dtype; how many it is goes by the lengths, on the device).
 * The workspace of the plan (0 bytes where no range is split) belongs to one call at a
 * time; for batches of several sizes it is the largest of their plans.  total_q *
 * num_q_heads < 2^31.
 * fp16 queries and outputs go to the tensor cores: codes are exact there, and a weight
 * times its token's scale is one fp16 number, held relative to the largest that its row
 * has met (in steps of 2^-29 of that one at most): half a step, 2^-11, of a weight, as the
 * output's own rounding is of the output.  fp32 queries or
 * outputs are computed in fp32 throughout, without the tensor cores, for small work.
 * A token whose codes or scale are not finite may make every output of its chunk NaN. */
kvq_status kvq_latent_plan(const kvq_latent* cache, int total_q, int num_seqs, int num_q_heads, int max_q_len,
                           int max_seq_len, int* num_splits, size_t* workspace_bytes);
kvq_status kvq_latent_attention(const kvq_latent* cache, const void* q, int total_q, const int32_t* cu_q_lens,
                                const int32_t* block_table, int max_pages, const int32_t* seq_lens, int num_seqs,
                                int num_q_heads, int max_q_len, int max_seq_len, int mode, float softmax_scale,
                                int causal, void* out, int out_dtype, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Expanded attention of ragged prompts, or of the last tokens of longer contexts, over
 * dense keys and values of each head (head_dim 128 and the shared rotary part; values of
 * 128).  With n keys of a sequence, query i of its m stands at n - m + i; causal as above:
 *   s_t = softmax_scale (q[0..128) . k_t + q[128..128+R) . r_t),  out = sum softmax(s)_t v_t
 *  q            [total_q][num_q_heads][128 + rope_dim], dense
 *  k, v         [128] of head h of row j at k + j * k_stride + h * k_head_stride (v likewise):
 *               slices of one projection's rows; strides in elements, multiples of 16 bytes
 *  k_rope       [rope_dim] of row j at k_rope + j * k_rope_stride
 *  cu_q_lens, cu_k_lens  device int32 [num_seqs + 1]: a sequence's rows of q, and of k, v and
 *               k_rope.  A sequence whose entries are not ascending ranges of at most max_q_len
 *               and max_k_len rows inside [0, total_q] and [0, total_k] is skipped and sets
 *               KVQ_DEVERR_QUERY_RANGE in the cache's error word.
 *  out          [total_q][num_q_heads][128], out_dtype;  lse as above
 * All device pointers, io_dtype of `cache`, whose pages are not read.  Queries that see no
 * key, other rows and the two ways of computing are as for kvq_latent_attention. */
typedef struct {
  const void* q;
  const void* k;
  const void* k_rope;
  const void* v;
  int64_t k_stride, k_head_stride;
  int64_t v_stride, v_head_stride;
  int64_t k_rope_stride;
  const int32_t* cu_q_lens;
  const int32_t* cu_k_lens;
  void* out;
  float* lse;
  int32_t total_q, total_k, num_seqs, num_q_heads, max_q_len, max_k_len;
  int32_t causal, out_dtype;
  float softmax_scale;
} kvq_latent_prompt;
kvq_status kvq_latent_prompt_attention(const kvq_latent* cache, const kvq_latent_prompt* p, void* stream);

/* ---- KVarN open tiles ---------------------------------------------------
 * [P2] 注意事项: a KVarN tile is exactly one 128-token page, and the backend
 * keeps a small fixed decode workspace.  A sequence's last, incomplete tile is
 * therefore held raw in a caller-owned tail buffer until its 128th token
 * arrives, when it is quantized into its page; decode reads the quantized
 * tiles plus the raw tail rows.
 *
 * Tail buffer (device, caller-owned, io_dtype): K rows [num_seqs][128][Hkv][D]
 * followed by V rows of the same shape; row r of sequence b holds token
 * 128 * floor(seq_len_b / 128) + r of that sequence, as written. */
kvq_status kvq_kvarn_tail_bytes(const kvq_cache* cache, int num_seqs, size_t* bytes);

/* Append tokens to their sequences' open tiles.  Token i (k, v [num_tokens][Hkv][D])
 * belongs to sequence seq_ids[i] at slot slot_mapping[i] = 128 * page + r: it is
 * copied to row r of that sequence's tail, and if r == 127 the tile is complete
 * and the sequence's 128 tail rows are quantized into `page` exactly as a
 * whole-tile kvq_quantize_write would.  Within one call a sequence's tokens
 * must belong to one tile (a decode step appends one token per sequence; a
 * prefill writes its whole tiles with kvq_quantize_write and appends the rest);
 * a tile completed by a call that also carries rows of another tile of the
 * same sequence is not written and sets KVQ_DEVERR_PARTIAL_TILE (its rows may
 * already be overwritten in the tail).  A negative
 * slot skips the token; a slot past the pool (KVQ_DEVERR_SLOT_RANGE) or a
 * seq_id outside [0, num_seqs) (KVQ_DEVERR_SEQ_ID) skips it and flags it.
 * Cache mode must be KVQ_KVARN_K4V2_G128; `tail` is 16-byte aligned and at
 * least kvq_kvarn_tail_bytes(num_seqs). */
kvq_status kvq_kvarn_append(kvq_cache* cache, const void* k, const void* v, const int32_t* slot_mapping,
                            const int32_t* seq_ids, int num_tokens, void* tail, int num_seqs, void* stream);

/* KVarN decode over whole tiles plus each sequence's open tile: any seq_len;
 * its first seq_len - seq_len % 128 tokens are read from the quantized pages
 * (as kvq_decode_attention does) and the last seq_len % 128 from rows 0.. of
 * the sequence's tail (raw, in the input domain).  The tail must hold
 * num_seqs sequences.  Workspace: kvq_kvarn_decode_workspace_bytes (never 0:
 * the tail is merged with the tiles' partial results by a second kernel). */
kvq_status kvq_kvarn_decode_workspace_bytes(const kvq_cache* cache, int num_seqs, int num_q_heads,
                                            int max_seq_len, size_t* bytes);
kvq_status kvq_kvarn_decode_attention(const kvq_cache* cache, const void* q, const int32_t* block_table,
                                      int max_pages, const int32_t* seq_lens, int num_seqs, int num_q_heads,
                                      int max_seq_len, float softmax_scale, const void* tail, void* out,
                                      int out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Tensor-level quantization error ([P5] "量化误差该怎样测", 张量层: MSE and
 * normalised MSE, max absolute error, cosine similarity, zero ratio,
 * clipping/saturation ratio, scale distribution, by head; K and V counted
 * separately).  For each token i with slot_mapping[i] >= 0 and each kv head,
 * the row the pool holds at that slot is dequantized and compared with the
 * row k[i] (v[i]) it was written from (KVarN rows are rotated back to the
 * input domain first).  dev_stats is a device array [2][num_kv_heads]
 * (index side * num_kv_heads + head, side 0 = K), zeroed by the call and then
 * accumulated; derived ratios are the caller's (e.g. NMSE = sum_sq_err /
 * sum_sq_ref, cosine = dot / sqrt(sum_sq_ref * sum_sq_deq)).  A slot past the
 * pool is skipped (KVQ_DEVERR_SLOT_RANGE).  Rows must have been written
 * (KVarN: whole tiles).  Diagnostic, not on the decode path. */
typedef struct {
  double count;           /* values compared */
  double sum_sq_err;      /* sum (x^ - x)^2 */
  double sum_sq_ref;      /* sum x^2 */
  double sum_sq_deq;      /* sum x^^2 */
  double dot;             /* sum x x^ */
  double max_abs_err;     /* max |x^ - x| */
  double zeros;           /* x^ == 0 */
  double saturated;       /* code at the largest magnitude of its grid (KVarN: the largest code) */
  double clipped;         /* saturated and |x| beyond |x^| by more than half the grid's last step
                             (INT8, INT4: s/2; E4M3: 16 s; NVFP4: one s_t s_b; KVarN: never) */
  double scale_hist[64];  /* stored scales by floor(log2 s) + 32, clamped to [0, 63]: per-token-head
                             and KVarN value scales once per row, NVFP4 block scales, KVarN key
                             scales once per tile (at its row 0), the per-tensor scale once per row */
} kvq_error_stats;
kvq_status kvq_tensor_error_stats(const kvq_cache* cache, const void* k, const void* v, const int32_t* slot_mapping,
                                  int num_tokens, kvq_error_stats* dev_stats, void* stream);

/* Allocation-free variant of kvq_decode_attention.  (No counterpart on the
 * source pages: this is an interface for callers, not part of the method.)
 * It is for callers that cannot allocate device memory when they decode --
 * for example code running inside a memory pool that was sized and frozen in
 * advance, or a host process embedding the library without any device
 * allocator of its own -- and so cannot provide the split-KV workspace.
 * Arguments and results are those of kvq_decode_attention minus the
 * workspace: the split partials go to a scratch array built into the library,
 * KVQ_NOALLOC_SCRATCH_BYTES bytes of device memory that every GPU loading the
 * library holds until the process exits.
 *  - A decode whose plan (kvq_decode_plan) needs more scratch than that is
 *    rejected with KVQ_ERR_CAPACITY before anything is launched.
 *  - The call allocates nothing: no cudaMalloc, no cudaFree, no allocating
 *    library routine.
 *  - The first call on a device looks up the array's device address (with
 *    that device current) and caches it; make that first call before any
 *    stream capture.
 *  - All calls share the one array and it keeps the last call's contents;
 *    calls whose kernels overlap on the GPU (different streams, or other
 *    host threads) race on it and must be serialised by the caller.
 *  - Each call writes every scratch entry it reads, so nothing has to be
 *    cleared between calls. */
#define KVQ_NOALLOC_SCRATCH_BYTES (32u << 20)
kvq_status kvq_decode_attention_noalloc(const kvq_cache* cache, const void* q, const int32_t* block_table,
                                        int max_pages, const int32_t* seq_lens, int num_seqs, int num_q_heads,
                                        int max_seq_len, int mode, float softmax_scale, void* out,
                                        int out_dtype, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KVQ_H */
