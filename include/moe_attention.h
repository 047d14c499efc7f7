/*
 * moe_attention.h — C ABI of the attention operators that stand beside the MoE
 * layer of a decoder block (NVIDIA GB300, sm_103a): norm and rotary positions of
 * the query and key heads, attention over packed sequences with its backward,
 * appending to a paged key/value cache, and attention of the newest tokens over
 * that cache.
 *
 * Conventions (pointers, streams, errors, ownership) are those of moe.h. Beside
 * them:
 *   - Heads: Hq query heads, Hkv key/value heads, Hq a multiple of Hkv; query
 *     head h reads key/value head h / G, G = Hq / Hkv. D values per head.
 *   - A moe_heads names the value (token t, head h, i) of a bf16 array at
 *     data[t * token_stride + h * head_stride + i]: strides are in elements, so
 *     the heads can be read in place from a fused projection or from a
 *     head-major array. Both strides are multiples of 8 and at least D wherever
 *     there is more than one token (head); an output's elements must not
 *     overlap. Data is 16-byte aligned.
 *   - Supported: D a multiple of 8, 8 <= D <= 128; G <= 64; Hq <= 1024; at most
 *     2^24 tokens. Zero tokens are allowed: the call does nothing (gradients of
 *     the norm weights are written as zeros).
 *   - Packed sequences: cu [B + 1] int32 on the device, cu[0] = 0, ascending;
 *     sequence b holds rows cu[b] .. cu[b + 1]. Sequences may be empty. Rows past
 *     cu[B] belong to no sequence; they are neither read nor written.
 *   - What only the device can see (offsets that do not ascend or pass the
 *     arrays, a sequence longer than the stated bound, a position outside the
 *     rotary table, a slot or page outside the cache) sets MOE_ERR_BAD_INDEX in
 *     the status word. Results of the row or sequence concerned are undefined (of
 *     every sequence that shares rows with another, where offsets do not ascend);
 *     a weight gradient is the sum without the row. All other results of the call
 *     are what they are without it, and later calls of this header run too: only
 *     after another error do they nothing. (The layer's calls do nothing after any,
 *     see moe.h.) Nothing is read or written out of bounds.
 *   - Sums, softmax statistics and norms are fp32; results are rounded once to
 *     bf16. Where a product runs on the tensor cores, the softmax weights and
 *     their gradients are its bf16 operands. Every result is the same from run to
 *     run (no floating-point atomics).
 *   - The attention kernels use programmatic stream serialization as the grouped
 *     GEMMs do (MOE_PDL); stream order holds as for ordinary launches.
 */
#ifndef MOE_ATTENTION_GB300_H
#define MOE_ATTENTION_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t Hq, Hkv, D;
} moe_attn_shape;

typedef struct {
    void* data; /* bf16 */
    int64_t token_stride, head_stride;
} moe_heads;

enum moe_rope_layout {
    MOE_ROPE_HALF = 0,       /* pairs (i, i + dims / 2)  */
    MOE_ROPE_INTERLEAVED = 1 /* pairs (2 i, 2 i + 1)     */
};

/* Rotary positions of the first `dims` values of a head (even, <= D; 0: none).
 * table [positions][dims / 2][2] fp32 holds (cos, sin), as moe_rope_table writes. */
typedef struct {
    const float* table;
    int32_t positions, dims, layout;
} moe_rope;

/* Paged cache: k, v [pages][Hkv][page_size][D] bf16, page_size a power of two in
 * [8, 256], pages * Hkv * page_size < 2^31. Token slot s is row s % page_size of
 * page s / page_size. */
typedef struct {
    void *k, *v;
    int32_t pages, page_size;
} moe_kv_cache;

/* table[p][i] = scale * (cos, sin)(p * inv_freq[i]), p < positions, i < dims / 2.
 * inv_freq is fp64 on the device and the angle is formed in fp64, so late
 * positions keep their precision; a long-context scaling of the frequencies is
 * whatever inv_freq and scale hold. */
int moe_rope_table(int32_t positions, int32_t dims, const double* inv_freq, double scale,
                   float* table, void* stream);

/* Per head of q [T, Hq, D] and k [T, Hkv, D]:
 *   y = x * (mean(x^2) + eps)^(-1/2) * w      (w = wq or wk, fp32 [D]; NULL: y = x)
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)    for the rotated pairs
 * with cos, sin of positions[t]. y is not rounded between the two steps. k may
 * have NULL data (only q). Outputs may be the inputs themselves. wq and wk are
 * both given or both NULL; positions may be NULL when rope.dims is 0. */
int moe_norm_rope(moe_attn_shape a, int32_t T, moe_heads q, moe_heads k, const float* wq,
                  const float* wk, float eps, const int32_t* positions, moe_rope rope,
                  moe_heads q_out, moe_heads k_out, void* stream);

/* Backward of moe_norm_rope from the gradients of its outputs and its inputs q, k
 * (nothing else is saved): dq, dk bf16 and dwq, dwk [D] fp32 (not written when the
 * weights are NULL). dq and dk may be dq_out and dk_out themselves. Gradients are
 * written, not accumulated. */
size_t moe_norm_rope_workspace_size(moe_attn_shape a, int32_t T);
int moe_norm_rope_backward(moe_attn_shape a, int32_t T, moe_heads dq_out, moe_heads dk_out,
                           moe_heads q, moe_heads k, const float* wq, const float* wk, float eps,
                           const int32_t* positions, moe_rope rope, moe_heads dq, moe_heads dk,
                           float* dwq, float* dwk, void* ws, size_t ws_bytes, void* stream);

/* moe_norm_rope of T new tokens whose keys go, with the values v, into row
 * slots[t] (int64) of the cache; the queries go to q_out. A token with a negative
 * slot is not stored. Slots of one call are distinct. */
int moe_kv_append(moe_attn_shape a, int32_t T, moe_heads q, moe_heads k, moe_heads v,
                  const float* wq, const float* wk, float eps, const int32_t* positions,
                  moe_rope rope, const int64_t* slots, moe_heads q_out, moe_kv_cache cache,
                  void* stream);

/* The sequences of moe_attention_*: B of them, cu_q over Tq query tokens, cu_k
 * over Tk key tokens, none longer than max_q and max_k. causal: query i of a
 * sequence with n queries and m keys sees the keys j <= i + m - n (the last query
 * sees them all); a query that sees no key gets out = 0, lse = -inf and no
 * gradient. Else every query sees every key of its sequence. */
typedef struct {
    int32_t B, Tq, Tk, max_q, max_k, causal;
    const int32_t *cu_q, *cu_k;
} moe_packed;

/* out [Tq, Hq, D] = softmax(scale q k^T) v per sequence and head, and
 * lse [Tq, Hq] fp32 = log sum exp(scale q k^T) (natural logarithm). scale > 0. */
int moe_attention_forward(moe_attn_shape a, moe_packed s, float scale, moe_heads q, moe_heads k,
                          moe_heads v, moe_heads out, float* lse, void* stream);

/* Gradients of moe_attention_forward from dout and its inputs and outputs. With
 * P = exp(scale q k^T - lse), dP = dout v^T, delta = sum_j P_j dP_j = sum_i dout_i out_i
 * and dS = P (dP - delta): dv = P^T dout, dq = scale dS k, dk = scale dS^T q, where dk
 * and dv sum over the G query heads of their head. Written, not accumulated; a
 * non-finite value of a sequence reaches no other sequence. */
size_t moe_attention_backward_workspace_size(moe_attn_shape a, moe_packed s);
int moe_attention_backward(moe_attn_shape a, moe_packed s, float scale, moe_heads dout,
                           moe_heads q, moe_heads k, moe_heads v, moe_heads out,
                           const float* lse, moe_heads dq, moe_heads dk, moe_heads dv, void* ws,
                           size_t ws_bytes, void* stream);

/* Attention of the newest n tokens of B sequences over the paged cache (their own
 * keys and values already in it). q, out: [B * n, Hq, D], rows b * n .. b * n + n
 * of sequence b; kv_lens [B] int32 counts its cached tokens, at most max_kv (no
 * more than 2^30); token t lies in row t % page_size of page
 * block_table[b * table_stride + t / page_size] (int32; entries past a sequence's
 * pages are not read). Query i sees
 * the tokens j <= i + kv_lens[b] - n; one that sees none gets zeros. The keys are
 * split over CTAs where B, Hkv and n leave the GPU idle, and the parts joined in a
 * fixed order. */
size_t moe_attention_decode_workspace_size(moe_attn_shape a, int32_t B, int32_t n, int32_t max_kv);
int moe_attention_decode(moe_attn_shape a, int32_t B, int32_t n, int32_t max_kv, float scale,
                         moe_heads q, moe_kv_cache cache, const int32_t* block_table,
                         int32_t table_stride, const int32_t* kv_lens, moe_heads out, void* ws,
                         size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_ATTENTION_GB300_H */
