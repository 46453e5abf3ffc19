/*
 * nvfp4_kv_cache.h -- C ABI of the NVFP4 key/value cache: appending to it and
 * attention over it (GB300, sm_103a).
 *
 * The conventions of nvfp4_router.h hold: device pointers owned by the caller,
 * asynchronous stream-ordered calls that never allocate, synchronise or copy
 * to the host (CUDA-graph capturable), arguments checked on the host before
 * any launch, nvr_status results, caller-allocated 256-byte aligned workspace
 * zeroed once.  Device-side values the host cannot check (slots, positions,
 * page ids, lengths) never cause an access outside the given arrays; what each
 * does when it is out of range is stated below.
 *
 * Cache layout
 * ------------
 * The cache is [n_pages, Hkv, page_bytes] uint8, page_bytes =
 * page_size * D * 9 / 8, 16-byte aligned.  One page of one KV head holds
 * page_size tokens of that head, contiguously (one bulk copy):
 *   key codes     [page_size][D/2]                 E2M1, element 2j in the low nibble
 *   key scales    [page_size][D/16]                E4M3, one per 16 channels
 *   value codes   [page_size/8][D/16][8 tokens][8 bytes]
 *   value scales  [page_size/8][D/16][8 tokens]
 * The value codes are transposed at the granularity of (8 tokens, 16
 * channels) so that a lane of the attention kernel gets two tokens of one
 * scale block with one 16-byte load.  An entry stands for
 * code * scale * gsa[head], with one fp32 global scale per KV head for keys
 * (k_gsa) and one for values (v_gsa): fixed when the cache is made, because
 * entries of many calls share them.  page_size is 16, 32, 64 or 128 and D
 * (channels per head) 64 or 128.  Slot s of the cache is token s % page_size
 * of page s / page_size.
 */
#ifndef NVFP4_KV_CACHE_H
#define NVFP4_KV_CACHE_H

#include "nvfp4_router.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one page of one KV head (0 for an unsupported page_size or D). */
size_t nvfp4_kv_page_bytes(int page_size, int D);

/*
 * nvfp4_kv_append -- for every token: RMS norm of each query and key head,
 * rotary positions, and the token's keys and values quantized into the cache.
 *
 *   q, k, v      [T, Hq, D], [T, Hkv, D], [T, Hkv, D] bf16 or fp32 (dt), heads
 *                contiguous, tokens *_stride elements apart (views of one fused
 *                projection, for instance); 16-byte aligned, strides multiples
 *                of 16 bytes.  Hq == 0 (q, q_out NULL) appends only.
 *   positions    [T] int32 rows of cos and sin
 *   slots        [T] int32 cache slots; a slot outside the cache stores nothing
 *                (the usual -1 of a padding token).  Two tokens with the same
 *                slot leave it unspecified.
 *   cos, sin     [n_pos, rot/2] fp32, 16-byte aligned
 *   rot          rotated channels, the first `rot` of a head: even, 0..D.
 *   interleaved  0: channel i pairs with i + rot/2; 1: 2i pairs with 2i + 1
 *   q_weight, k_weight  [D] fp32 or NULL (no norm of that side)
 *   q_out        out [T, Hq, D] bf16; must not overlap q, k or v
 * Arithmetic, fp32 rounded to nearest at every step so that the stored bits are
 * a function of the inputs alone:
 *   x *= 1 / sqrt(sum(x^2) / D + eps), then x *= weight; the sum halves the
 *     head repeatedly (channel i + channel i + D/2, then + D/4, ...);
 *   (a, b) -> (a cos - b sin, b cos + a sin);
 *   queries: rounded once to bf16; keys (after the rotation) and values: the
 *   quantizer of nvfp4_quantize_act with gsa in place of the call's own scale
 *   (magnitudes above 2688 gsa saturate).
 * A position outside [0, n_pos) zeroes the token's q_out row and stores
 * nothing.  One kernel, no workspace.
 */
nvr_status nvfp4_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, nvr_dtype dt, int64_t T, int Hq, int Hkv, int D,
                           const int32_t* positions, const int32_t* slots, const float* cos, const float* sin,
                           int64_t n_pos, int rot, int interleaved, const float* q_weight, const float* k_weight,
                           float eps, const float* k_gsa, const float* v_gsa, uint8_t* cache, int64_t n_pages,
                           int page_size, void* q_out, nvr_stream_t stream);

/*
 * nvfp4_kv_gather -- the values that n slots stand for: k_out and v_out
 * [n, Hkv, D], bf16 or fp32 (out_dt), code * scale * gsa rounded to fp32, and for
 * bf16 from there; zeros for a slot outside the cache.  One kernel, no workspace.
 */
nvr_status nvfp4_kv_gather(const uint8_t* cache, int64_t n_pages, int page_size, int Hkv, int D,
                           const int32_t* slots, int64_t n, const float* k_gsa, const float* v_gsa, void* k_out,
                           void* v_out, nvr_dtype out_dt, nvr_stream_t stream);

/*
 * nvfp4_kv_attention -- softmax attention of new queries over the cached keys
 * and values of their sequences:
 *   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale * q . k_t)
 * Query head h reads KV head h / (Hq / Hkv).  Query i of the m queries of a
 * sequence with n cached tokens (its own among them) has position n - m + i;
 * with `causal` it sees the tokens up to that position, with window > 0 (causal
 * only) the last `window` of them.
 *
 *   q            [T, Hq, D] bf16, heads contiguous, tokens q_stride elements
 *                apart (16-byte aligned, q_stride a multiple of 8)
 *   page_table   [B, max_pages] int32: sequence b's token t lies in page
 *                page_table[b, t / page_size]; entries past its length are
 *                not used (some are read, inside the table); tokens of a page
 *                id outside [0, n_pages) are not seen
 *   kv_lens      [B] int32, taken within [0, max_pages * page_size]
 *   cu_q         [B + 1] int32: sequence b's queries are rows
 *                cu_q[b]..cu_q[b + 1] of q, at most max_q of them; or NULL: every
 *                sequence has max_q queries (T == B * max_q).  Values are taken within
 *                [0, T] and must not decrease (else some rows are unspecified).  Rows that
 *                no sequence covers (in front of the first one, behind the last one, past
 *                max_q in one) get zeros and lse = -inf; rows past max_q count as
 *                queries for the positions of those in front of them.
 *   out          out [T, Hq, D] bf16, 16-byte aligned
 *   lse          out [T, Hq] fp32 or NULL: log sum_t exp(scale * q . k_t)
 *   workspace    nvfp4_kv_attention_workspace_size(...) bytes, zeroed once
 * Calls whose work does not fit 31 bits (B * Hkv * columns / 16 * tokens of the page
 * table's width / 128) are NVR_ERR_UNSUPPORTED.
 * A query that sees no token gets zeros and lse = -inf, one with a NaN among its
 * channels NaNs in both.  What the cache holds of tokens that no query sees (any
 * bytes: past the length, in front of the first window, in the same page as seen
 * ones or not) does not reach the output; a NaN in a key's or value's scales
 * reaches the queries that see the token, no others.  Hq is a multiple of Hkv.
 * Scores, softmax statistics and outputs are accumulated in fp32; the weights p_t
 * enter the second product as fp16, relative to a running maximum (a weight below
 * 2^-32 of the largest is lost there); results do not depend on the order in which
 * the GPU runs the blocks.  One kernel and, unless no key can be cut over blocks, a
 * second one that joins the parts of those that were.  The workspace's size depends
 * on D alone (T_max, B_max and the heads are checked): partial results of the
 * resident blocks.  A bounded wait that runs out sets the workspace's status word
 * (nvr_read_device_status).
 */
size_t nvfp4_kv_attention_workspace_size(int64_t T_max, int64_t B_max, int Hq, int Hkv, int D);
nvr_status nvfp4_kv_attention(const void* q, int64_t q_stride, int64_t T, int Hq, int Hkv, int D,
                              const uint8_t* cache, int64_t n_pages, int page_size, const int32_t* page_table,
                              int64_t B, int64_t max_pages, const int32_t* kv_lens, const int32_t* cu_q, int max_q,
                              const float* k_gsa, const float* v_gsa, float scale, int causal, int window,
                              void* out, float* lse, void* workspace, size_t ws_bytes, nvr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_KV_CACHE_H */
