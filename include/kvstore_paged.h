/*
 * libkvstore -- operators on a paged K/V cache, beside the stores of
 * kvstore.h: rotated append, load, and attention.
 *
 * The conventions are those of kvstore.h: every pointer is a DEVICE pointer
 * owned by the caller (except the two structs' own addresses, which are host
 * pointers read during the call), strides are in bytes unless stated, work is
 * enqueued on the given stream of the current device, nothing is allocated,
 * freed or waited for, so every call may be captured into a HIP graph, and
 * negative codes mean that nothing was launched (but for KVSTORE_ERR_HIP from
 * a later launch of a call that needs several).
 *
 * A paged cache holds slots of num_heads x head_dim elements; slot s lies in
 * page s / page_size at offset s % page_size.  Its element formats:
 *
 *   KVSTORE_FMT_BF16, _FP16   the 16-bit values themselves;
 *   KVSTORE_FMT_E4M3FN, _E5M2 8-bit codes; a value is code * scale, the scale
 *                             fp32 and one for the tensor, for each token, or
 *                             for each token and head;
 *   KVSTORE_FMT_FP4           4-bit e2m1 codes (1 sign, 2 exponent, 1 mantissa
 *                             bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte,
 *                             the even element in the low half, with one scale
 *                             byte (e8m0: 2^(byte - 127), 255 is NaN) for each
 *                             block of 32 elements of a head.
 *
 * Out-of-range slots, positions and pages never fault: what they name is
 * skipped and recorded in the error flag of kvstore.h (kvstore_check_error,
 * kvstore_take_error).
 */
#ifndef KVSTORE_PAGED_H
#define KVSTORE_PAGED_H

#include "kvstore.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element formats of a paged cache. */
enum {
  KVSTORE_FMT_BF16 = 0,
  KVSTORE_FMT_FP16 = 1,
  KVSTORE_FMT_E4M3FN = 2,
  KVSTORE_FMT_E5M2 = 3,
  KVSTORE_FMT_FP4 = 4
};

/* Where a reader finds the scales of an FP8 or 4-bit cache. */
enum {
  KVSTORE_SCALES_TENSOR = 0,     /* one fp32 each at k_scales / v_scales; NULL: 1.0 */
  KVSTORE_SCALES_TOKEN = 1,      /* fp32 at page and offset strides */
  KVSTORE_SCALES_TOKEN_HEAD = 2, /* fp32 at page, offset and head strides */
  KVSTORE_SCALES_BLOCK = 3       /* e8m0 bytes at page, offset and head strides, then
                                    one byte for each block of 32 elements */
};

/*
 * A K and a V cache of one shape.  Element d of head h of slot (page, off)
 * lies at byte page * *_stride_page + off * *_stride_offset + h *
 * *_stride_head of the cache, plus 2 * d (16 bits), d (FP8) or d / 2 (4
 * bits).  Strides >= 0, caches and cache strides 16-byte aligned (a head of
 * 4-bit elements: head strides of a multiple of 16), fp32 scales and their
 * strides 4-byte aligned.  head_dim is a multiple of 16 (4 bits: of 32) of
 * at most 512; page_size and num_heads > 0; slots are [0, num_slots).
 * scale_kind: TENSOR for 16-bit caches (no scales are read), TENSOR, TOKEN or
 * TOKEN_HEAD for FP8, BLOCK for 4 bits.
 */
typedef struct kvstore_paged_cache {
  void* k;
  void* v;
  int32_t format;
  int32_t scale_kind;
  int32_t num_heads;
  int32_t head_dim;
  int64_t page_size;
  int64_t num_slots;
  int64_t k_stride_page, k_stride_offset, k_stride_head;
  int64_t v_stride_page, v_stride_offset, v_stride_head;
  void* k_scales;
  void* v_scales;
  int64_t ks_stride_page, ks_stride_offset, ks_stride_head;
  int64_t vs_stride_page, vs_stride_offset, vs_stride_head;
} kvstore_paged_cache;

/* The rows of kvstore_rope_paged: *[t, h, d] at t * *_stride_token + h *
 * *_stride_head + 2 * d, 16-byte aligned, strides >= 0. */
typedef struct kvstore_rope_rows {
  const void* q;   /* NULL: no q (q_heads is not read) */
  void* q_out;     /* may be q itself, with the same strides */
  const void* k;
  const void* v;
  int32_t src_dtype; /* KVSTORE_SRC_BF16 / KVSTORE_SRC_FP16 */
  int32_t q_heads;
  int64_t q_stride_token, q_stride_head;
  int64_t qo_stride_token, qo_stride_head;
  int64_t k_stride_token, k_stride_head;
  int64_t v_stride_token, v_stride_head;
} kvstore_rope_rows;

/*
 * Rotates q and k by their tokens' positions and writes k and v into their
 * cache slots, in one pass.
 *
 * Rotation of the first rot_dim dims of a head, at position p, with c_i =
 * cos_sin[p][i] and s_i = cos_sin[p][rot_dim / 2 + i], for each pair (a, b) =
 * (x_i, x_{i + rot_dim/2}), or (x_2i, x_{2i+1}) if interleaved:
 *   a' = a * c_i - b * s_i,   b' = b * c_i + a * s_i,
 * in fp32, every product, sum and difference rounded to nearest on its own.
 * Dims from rot_dim on, and v, stay as they are.  q_out is rounded once to
 * the source type; k' and v go into the cache:
 *   16 bits  rounded to the format, which must be the source type;
 *   FP8      x * inv (inv_k_scale_ptr / inv_v_scale_ptr: one fp32 each, NULL:
 *            1.0), rounded, saturated and NaN-coded as in kvstore_fp8_paged;
 *            scale_kind must be KVSTORE_SCALES_TENSOR, and the cache's own
 *            scale pointers are not read;
 *   4 bits   per block of 32: scale = the smallest power of two >= 2^-100 with
 *            max |x| <= 7 * scale, so that the largest element rounds by no
 *            more than the format's own half step; elements to the nearest
 *            e2m1 value of x / scale, ties to the even code, beyond 6 to 6; a
 *            block with a NaN or infinity gets the NaN scale.
 *
 *   positions   [batch], contiguous, of type pos_dtype (KVSTORE_IDX_*), each
 *               in [0, num_positions).
 *   cos_sin     [num_positions] rows of rot_dim fp32 at cos_sin_stride bytes;
 *               16-byte aligned.  NULL (with positions NULL): no rotation.
 *   rot_dim     a multiple of 16, at most head_dim.
 *   indices, idx_dtype, idx_stride, batch: as in kvstore_copy.
 *
 * A token whose slot is outside [0, num_slots) is recorded, its k and v are
 * not written, its q is.  A token whose position is out of range is recorded
 * and nothing of it is written.  Slots must be unique within a call.
 */
int kvstore_rope_paged(const kvstore_rope_rows* rows, const void* positions, int pos_dtype,
                       const float* cos_sin, int64_t cos_sin_stride, int64_t num_positions,
                       int32_t rot_dim, int interleaved, const void* indices, int idx_dtype,
                       int64_t idx_stride, const kvstore_paged_cache* cache,
                       const float* inv_k_scale_ptr, const float* inv_v_scale_ptr, uint32_t batch,
                       hipStream_t stream);

/*
 * Reads the rows of slots indices[t] out of a cache: k_out[t, h, d] =
 * dst_dtype(value), with the value in fp32 (code * scale, one rounding) and
 * rounded once to dst_dtype (KVSTORE_SRC_*).  k_out / v_out: 16-byte aligned,
 * strides too.  A token whose slot is out of range is recorded and its rows
 * are left as they were.  16-bit caches must be of type dst_dtype (their bits
 * are copied).
 */
int kvstore_load_paged(const kvstore_paged_cache* cache, const void* indices, int idx_dtype,
                       int64_t idx_stride, void* k_out, int64_t ko_stride_token,
                       int64_t ko_stride_head, void* v_out, int64_t vo_stride_token,
                       int64_t vo_stride_head, int dst_dtype, uint32_t batch, hipStream_t stream);

/*
 * Attention of new tokens over cached sequences.
 *
 * Sequence b has seq_lens[b] keys (negative: 0; above max_pages * page_size:
 * that), the last of them those of its own new tokens, which are the rows
 * cu_q[b] ... cu_q[b + 1] - 1 of q (cu_q NULL: row b alone).  The new token r
 * of n has position p = seq_lens[b] - n + r and sees the keys
 *   k <= p   with   p - k < window  or  k < sinks
 * (window 0: all k <= p).  Key k lies in page page_table[b * table_stride + k
 * / page_size] at offset k % page_size.  For q head h, with kv head h /
 * (q_heads / num_heads):
 *   out = sum_k softmax_k(sm_scale * q . K_k) V_k,   0 where no key is seen
 * (or where every score is -infinity).
 * Keys that a row does not see never reach it, whatever their slots hold (NaN
 * and infinities included).  A page outside [0, num_slots / page_size) holds
 * no keys; the first row of every group of rows that meets it is recorded in
 * the error flag.  Rows of q before cu_q[0] and from cu_q[seqs] on are not
 * read and their out is left as it was.  cu_q must not decrease; values
 * outside [0, tokens] are taken as the nearer end.
 *
 * Arithmetic: q and the cached values are multiplied in the source type's
 * precision on the matrix cores with fp32 sums; FP8 and 4-bit values are
 * exact in it (with fp16 sources the values must lie in fp16's range);
 * softmax statistics and sums are fp32; the weights are rounded to the source
 * type for the product with V.
 */
typedef struct kvstore_attention_args {
  const void* q; /* [tokens, q_heads, head_dim], 16-byte aligned, strides too */
  void* out;     /* the same shape; must not overlap q */
  int64_t q_stride_token, q_stride_head;
  int64_t o_stride_token, o_stride_head;
  int32_t src_dtype;         /* KVSTORE_SRC_*: of q, out and 16-bit caches */
  int32_t q_heads;           /* a multiple of num_heads */
  const int32_t* cu_q;       /* [seqs + 1], or NULL (then tokens == seqs) */
  uint32_t tokens;           /* rows of q */
  uint32_t seqs;
  uint32_t max_q;            /* most new tokens of a sequence, if known; 0: tokens.
                                Steers the launch only */
  const int32_t* page_table; /* [seqs, max_pages] */
  int64_t table_stride;      /* in elements */
  uint32_t max_pages;        /* 0 < max_pages * page_size < 2^31 - 1024 */
  const int32_t* seq_lens;   /* [seqs] */
  int64_t max_len;           /* longest sequence, if known; 0: max_pages * page_size.
                                Steers the launch only */
  int64_t window;            /* >= 0 */
  int64_t sinks;             /* >= 0; not read if window is 0 */
  float sm_scale;            /* in [0, 2.3e38] */
  void* workspace;           /* kvstore_attention_workspace bytes, 16-byte aligned; in
                                use until the call's work is done */
  int64_t workspace_bytes;
} kvstore_attention_args;

/* Bytes of workspace that the call needs (0: none; the pointers of `args` and
 * `cache` are not read), or a negative status. */
int64_t kvstore_attention_workspace(const kvstore_attention_args* args,
                                    const kvstore_paged_cache* cache);

/* head_dim is at most 256 here, page_size below 2^31, and num_slots holds at
 * least one page. */
int kvstore_attention_paged(const kvstore_attention_args* args, const kvstore_paged_cache* cache,
                            hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVSTORE_PAGED_H */
