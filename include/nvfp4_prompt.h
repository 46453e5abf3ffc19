/*
 * nvfp4_prompt.h -- C ABI of a prompt's operators beside the NVFP4 key/value
 * cache: rotary positions with several axes, and attention of packed prompts over
 * their own 16-bit keys and values (GB300, sm_103a).
 *
 * The conventions of nvfp4_router.h hold: device pointers owned by the caller,
 * asynchronous stream-ordered calls that never allocate, synchronise or copy
 * to the host (CUDA-graph capturable), arguments checked on the host before
 * any launch, nvr_status results, caller-allocated 256-byte aligned workspace
 * zeroed once.  Device-side values the host cannot check (positions, offsets)
 * never cause an access outside the given arrays; what each does when it is out
 * of range is stated below.
 */
#ifndef NVFP4_PROMPT_H
#define NVFP4_PROMPT_H

#include "nvfp4_router.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PROMPT_ROPE_MAX_D 256
#define PROMPT_ROPE_MAX_PAIRS (PROMPT_ROPE_MAX_D / 2)
#define PROMPT_ROPE_MAX_AXES 8

/*
 * prompt_rope -- RMS norm of each query and key head and rotary positions with
 * several axes (time, height and width of a patch, for instance):
 *   x *= weight / sqrt(sum(x^2) / D + eps);  (a, b) -> (a cos - b sin, b cos + a sin)
 * where pair i of a head takes column i of row positions[axes[i]] of the tables.
 *
 *   q, k         [T, Hq, D], [T, Hkv, D] bf16, fp16 or fp32 (dt), heads contiguous,
 *                tokens *_stride elements apart.  Hq == 0 or Hkv == 0: only the other one.
 *   D            even, at most PROMPT_ROPE_MAX_D
 *   positions    [n_axes][T] int32, axes axis_stride elements apart
 *   axes         HOST array of rot/2 bytes: the axis of each pair, below n_axes
 *                (1 .. PROMPT_ROPE_MAX_AXES); read during the call
 *   cos, sin     [n_pos, rot/2] fp32
 *   rot          rotated channels, the first `rot` of a head: even, 0..D (0: norm only;
 *                positions, axes, cos and sin are not looked at)
 *   interleaved  0: channel i pairs with i + rot/2; 1: 2i pairs with 2i + 1
 *   q_weight, k_weight  [D] fp32 or NULL (no norm of that side)
 *   q_out, k_out out [T, Hq, D], [T, Hkv, D] of out_dt (dt, or bf16 or fp16 for fp32
 *                heads), tokens *_out_stride elements apart; each may be its input itself
 *                (same type and stride), must not overlap the inputs or the other result otherwise
 * fp32 arithmetic, rounded once to out_dt.  A token with a position outside
 * [0, n_pos) on an axis that some pair goes by gets zeros.  Fast for heads of 64, 128
 * and 256 channels that are 16-byte aligned (strides too), with rot a multiple of 16 (8
 * if interleaved); others are taken a channel at a time and take some 15 times as long.
 * fp16 heads are for prompts by themselves: nvfp4_kv_append takes bf16 and fp32 ones.  One
 * kernel, no workspace.
 */
nvr_status prompt_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, nvr_dtype dt, int64_t T,
                       int Hq, int Hkv, int D, const int32_t* positions, int64_t axis_stride, int n_axes,
                       const uint8_t* axes, const float* cos, const float* sin, int64_t n_pos, int rot,
                       int interleaved, const float* q_weight, const float* k_weight, float eps, void* q_out,
                       int64_t q_out_stride, void* k_out, int64_t k_out_stride, nvr_dtype out_dt,
                       nvr_stream_t stream);

/*
 * prompt_attention -- softmax attention of packed sequences of different lengths over
 * their own 16-bit keys and values:
 *   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale * q . k_t)
 * Query head h reads KV head h / (Hq / Hkv).  Query i of the m queries of a sequence
 * with n keys has position n - m + i; with `causal` it sees the keys up to that
 * position, with window > 0 (causal only) the last `window` of them.
 *
 *   q, k, v      [T, Hq, D], [Tk, Hkv, D], [Tk, Hkv, D] bf16 or fp16 (dt); tokens
 *                *_stride and heads *_head_stride elements apart, in any order (views of
 *                one fused projection, or heads outermost): at least D, multiples of
 *                16 bytes, below 2^38; 16-byte aligned.  D is 64 or 128.
 *   cu_q         [B + 1] int32: sequence b's queries are rows cu_q[b]..cu_q[b + 1] of q,
 *                at most max_q of them; or NULL: every sequence has max_q queries
 *                (T == B * max_q)
 *   cu_k         [B + 1] int32: the same for its keys and values, at most max_k of them;
 *                or NULL: those of its queries (Tk == T; max_k is not looked at)
 *                Values are taken within [0, T] or [0, Tk] and must not decrease (else rows
 *                are unspecified), nor change while the call runs.  Rows that no sequence covers (in front of the first
 *                one, behind the last one, past max_q in one) get zeros and lse = -inf; keys
 *                past max_k (without cu_k: past max_q) are not seen; both count for the
 *                positions.
 *   prefix_out, prefix_lse  [T, Hq, D] of dt, 16-byte aligned, and [T, Hq] fp32, or both
 *                NULL: the result of attention of the same queries over other keys (a cached
 *                prefix: nvfp4_kv_attention without `causal`, whose results are bf16), joined as if
 *                all keys had been seen at once.  A row whose prefix_lse is -inf has no
 *                prefix.  They may be out and lse themselves.
 *   scale        finite, and so that scale * log2(e) is (else NVR_ERR_INVALID_ARG)
 *   out          out [T, Hq, D] of dt, 16-byte aligned, must not overlap q, k or v
 *   lse          out [T, Hq] fp32 or NULL: log sum_t exp(scale * q . k_t)
 *   workspace    prompt_attention_workspace_size(...) bytes, zeroed once
 * A query that sees no key and has no prefix gets zeros and lse = -inf, one with a NaN
 * among its channels, or among those of a key that it sees, NaNs in both (with a scale of
 * zero too, and there with an infinity as well).  What lies in keys and values that a query
 * does not see (other sequences', later ones, those in front of the window: infinities and
 * NaNs among them) does not reach its result.
 * Scores, softmax statistics and outputs are accumulated in fp32; the weights p_t enter the
 * second product rounded to dt, relative to a running maximum (fp16: a weight below 2^-32
 * of the largest is lost there, and results within 2^-11 of fp16's largest value may become
 * infinite; bf16: results above 2^100 may overflow); results do not depend on the order in which
 * the GPU runs the blocks.  One kernel.
 * The rows (query, head) of a KV head are taken in pairs of tiles of up to 128 rows: s = 256 / G
 * queries a pair where G = Hq / Hkv is a power of two up to 128 (other G: about as many), at most
 * P = Hkv * min(B * ceil(max_q / s), T / s + B) pairs, each over n = ceil(max_k / 128) tiles of keys
 * at most, or those of the window.  Calls of P * (2 n + 5) >= 2^31 - 2^24, whatever a causal mask
 * hides, of B * ceil(max_q / s) >= 2^30, of B > 2^24, or of n > 2^18 with P (2 n + 5) >= 2^26 + 2^8
 * are NVR_ERR_UNSUPPORTED (one prompt of 64 query heads: from 738432 tokens on).  Room that max_q
 * and max_k leave above T and Tk does not count.
 * The workspace's size depends on D alone (the heads are checked): it holds partial results of the
 * resident blocks, of one call at a time.  A bounded wait that runs out sets its status word
 * (nvr_read_device_status); the workspace is to be zeroed again then.
 */
size_t prompt_attention_workspace_size(int Hq, int Hkv, int D);
nvr_status prompt_attention(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k, int64_t k_stride,
                            int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride,
                            nvr_dtype dt, int64_t T, int64_t Tk, int Hq, int Hkv, int D, const int32_t* cu_q,
                            const int32_t* cu_k, int64_t B, int max_q, int max_k, float scale, int causal, int window,
                            const void* prefix_out, const float* prefix_lse, void* out, float* lse, void* workspace,
                            size_t ws_bytes, nvr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_PROMPT_H */
