/*
 * k3moe_serve.h — the third part of libk3moe's C ABI: rows in microscaled 8
 * bits (rounding, the residual's addition with a root-mean-square norm, and
 * products with microscaled 4-bit weights), routing to experts by groups, and
 * the verification of drafted tokens.  Every general convention of k3moe.h
 * holds here too (device pointers, 16-byte alignment, caller-owned buffers,
 * host checks before anything is enqueued, status codes, outputs fully
 * overwritten, reentrancy).
 *
 * A microscaled 8-bit matrix [R, K] (K a multiple of 32) is a pair
 *   codes  u8 [R, K]     E4M3 codes: sign, four exponent bits (bias 7), three
 *                        mantissa bits; largest magnitude 448, 127 and 255 = NaN
 *   scale  u8 [R, K/32]  E8M0 byte e of each 32 elements: the value 2^(e-127),
 *                        255 = NaN
 */
#ifndef K3MOE_SERVE_H
#define K3MOE_SERVE_H

#include "k3moe_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mxfp8_quantize — float rows to microscaled 8 bits.
 * Source of the rounding: the OCP Microscaling Formats specification 1.0, as
 * for mxfp4_quantize; the pages keep the dense tensors around the experts in 8
 * bits and more (Hugging Face card "K3-Stuff", scripts list: a trunk in Q8_0).
 *
 *   x       [R, K] f32, bf16 or f16 (x_dtype)
 *   codes   u8 [R, K], scale u8 [R, K/32]: out
 *
 * Block scale 2^e with e = max(floor(log2 m) - 8, -127), m = the block's
 * largest magnitude; with saturate == 0, e is one larger where m > 448 * 2^e,
 * so that no element is clamped.  A code is the E4M3 value nearest to v / 2^e,
 * ties to the even code, magnitudes above 448 clamped to 448, the sign kept
 * (also of zeros).  An all-zero block has scale byte 0.  A block holding an
 * infinity or a NaN gets scale byte 255 and the code 127 for every element.
 * Sizes and statuses as mxfp4_quantize.
 */
int mxfp8_quantize(const void* x, int32_t x_dtype, int64_t R, int64_t K, int32_t saturate, uint8_t* codes,
                   uint8_t* scale, void* stream);

/*
 * mxfp8_unpack — the values of a microscaled 8-bit matrix: out [R, K] f32 or
 * bf16 (out_dtype), code * 2^(e-127), the sign of zero kept, NaN for a NaN code
 * or scale byte 255; exact, except that values beyond the largest finite number
 * become infinite and bf16 values below 2^-126 are rounded to its subnormals.
 * Sizes and statuses as mxfp4_unpack.
 */
int mxfp8_unpack(const uint8_t* codes, const uint8_t* scale, int64_t R, int64_t K, int32_t out_dtype, void* out,
                 void* stream);

/*
 * mxfp8_rms_norm — what stands between two layers: the residual's addition, a
 * root-mean-square norm, and the normed rows in microscaled 8 bits.
 * Source: llama.cpp pull request "model: add Kimi-K3 text model", dry-run
 * comment (norm tensors, ffn_routed_norm); the norm's epsilon is a hyperparameter.
 *
 *   v = x + residual                    (x where residual is NULL)
 *   y = v / sqrt(mean(v^2) + eps) * gamma
 *
 *   x, residual  [R, K] f32, bf16 or f16 (x_dtype); residual may be NULL
 *   gamma        [K] f32, bf16 or f16 (gamma_dtype), or NULL for ones
 *   sum          [R, K] of x_dtype, or NULL: out, v rounded once
 *   y            [R, K] of x_dtype, or NULL: out, y rounded once
 *   codes, scale the pair of mxfp8_quantize(y) with `saturate`: out, or both
 *                NULL where y is not
 *
 * v, the mean, y and its rounding to 8 bits are computed in fp64, so y's
 * codes are those of the exact y unless it lies within about 1e-15 of a
 * border between two codes, and neither sum's nor y's own rounding enters
 * them. y is rounded once from that fp64 value, subnormal results of its
 * type included. A row with a non-finite v, or (eps == 0) of zeros, gives
 * what that arithmetic gives: NaN, or zeros beside an infinity, and scale
 * bytes as mxfp8_quantize; so does a block with elements beyond 2^136.
 * sum may be x or residual itself (updated in place); else no output overlaps
 * an input or another output. Deterministic.
 * Sizes: as mxfp4_quantize, eps >= 0 (K3MOE_ERR_SHAPE). Unknown types:
 * K3MOE_ERR_UNSUPPORTED. codes without scale, scale without codes, or neither
 * and no y: K3MOE_ERR_NULL.
 */
int mxfp8_rms_norm(const void* x, const void* residual, const void* gamma, int32_t x_dtype, int32_t gamma_dtype,
                   int64_t R, int64_t K, double eps, int32_t saturate, void* sum, void* y, uint8_t* codes,
                   uint8_t* scale, void* stream);

/*
 * mxfp8_matmul — rows in microscaled 8 bits times a microscaled 4-bit weight
 * matrix,
 *   out[m][n] = sum_k A[m][k] * W[n][k],
 *   a_codes u8 [M, K], a_scale u8 [M, K/32]
 *   w_packed u8 [N, K/2], w_scale u8 [N, K/32], the layout of mxfp4_matmul
 *   out [M, N] f32 or bf16 (out_dtype)
 * Exact products of the stored values, summed in fp32 and rounded once for a
 * bf16 output. A NaN scale or code of A makes its row of out NaN, a NaN scale
 * of W its column. Deterministic.
 * Sizes and statuses as mxfp4_matmul.
 */
int mxfp8_matmul(const uint8_t* a_codes, const uint8_t* a_scale, const uint8_t* w_packed, const uint8_t* w_scale,
                 int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* out, void* stream);

/* Score functions of moe_route_groups. */
#define K3MOE_SCORE_SIGMOID 0
#define K3MOE_SCORE_SOFTMAX 1

/*
 * moe_route_groups — top-k routing within the best groups of experts.
 * Source: llama.cpp pull request "model: add Kimi-K3 text model", review
 * comment on the converter dry run (expert count, experts used, score gating
 * function, per-expert bias exp_probs_b). The groups are equal runs of
 * consecutive experts, as a deployment that keeps each group on one device
 * limits how many devices a token reaches; groups == 1 has none.
 *
 *   logits  f32 [T, E], bias f32 [E] or NULL for zero
 *   topk_ids i32 [T, k], topk_w f32 [T, k]: out, best first
 *
 * Gate g[t,e] = 1/(1+exp(-z)) (K3MOE_SCORE_SIGMOID) or exp(z) / sum_e'
 * exp(z) (K3MOE_SCORE_SOFTMAX), score s = g + b, evaluated in fp64 (a
 * softmax to about 2e-14 of itself: scores nearer than that, but of other
 * logits and biases, may rank either way). A group's score is the sum of its
 * group_top (1 or 2) best scores (of all, where it has fewer). The
 * topk_groups best groups are kept, and of their experts the k with the
 * highest scores are selected; the lower index goes first among equal
 * scores, of groups as of experts. A NaN score ranks below every number, as
 * -inf. The weight of a selected expert is its gate (the bias only steers
 * selection), divided by the sum over the k selected when `normalize` != 0
 * (0 where that sum is 0), times `route_scale`, rounded once to f32. NaN
 * logits leave the softmax of the others as it is without them; where logits
 * are +inf, they share it equally; where all are -inf, every gate is 0.
 * Sizes: 0 <= T <= 2^36 (T == 0 is a no-op), 1 <= E <= K3MOE_MAX_EXPERTS_FFN, groups
 * >= 1 divides E, 1 <= topk_groups <= groups, 1 <= k <= min(K3MOE_MAX_TOPK,
 * topk_groups * E / groups); K3MOE_ERR_SHAPE otherwise. Unknown score, or a
 * group_top other than 1 and 2: K3MOE_ERR_UNSUPPORTED.
 */
int moe_route_groups(const float* logits, const float* bias, int64_t T, int32_t E, int32_t groups, int32_t topk_groups,
                     int32_t group_top, int32_t k, int32_t score, int32_t normalize, float route_scale,
                     int32_t* topk_ids, float* topk_w, void* stream);

/* Largest vocabulary of moe_verify_draft. */
#define K3MOE_MAX_VOCAB (1 << 24)

/*
 * moe_verify_draft — speculative verification: which of the drafted tokens the
 * target accepts, and the token after them.
 * Source: lucebox pull request "feat(kimi-k3): add DSpark Q8 artifact and
 * shared speculative runtime", "DSpark acceptance-contract correction"
 * (verification is the current token plus 7 proposals: width 8). The pages do
 * not spell the rule out; it is the published one that keeps the target's
 * distribution: proposal x is accepted where u q(x) < p(x), and at the first one
 * that is not, the next token is drawn from max(p - q, 0), normalised.
 *
 *   logits       [S, W, V] f32, bf16 or f16 (dtype): row w of a sequence is the
 *                target's after position w (0: the current token, then the
 *                W - 1 proposals), in the row order of moe_verify_width_distinct
 *   draft_ids    i32 [S, W-1]     the proposals
 *   draft_probs  f32 [S, W-1, V]  q, the draft's distributions, or NULL: each
 *                                 proposal had probability 1
 *   draft_len    i32 [S] or NULL  proposals of each sequence (W - 1 where NULL;
 *                                 clamped to 0 .. W - 1)
 *   temperature  f32 [S] or NULL  p = softmax(logits / temperature); 1 where
 *                                 NULL; 0, below or NaN: greedy
 *   u_accept     f32 [S, W-1], u_sample f32 [S]  uniforms in [0, 1)
 *   n_accepted   i32 [S]    out: length of the accepted prefix
 *   tokens       i32 [S, W] out: the accepted proposals, the next token, then -1
 *   accept_prob  f32 [S, W-1] out, or NULL: min(1, p(x) / q(x)) of every
 *                proposal, 0 past draft_len (their means over sequences are what
 *                moe_verify_width_choose takes as `accept`)
 *
 * The next token is the lowest v whose cumulative probability (in index order)
 * exceeds u_sample times the total, of max(p - q, 0) at the first proposal that
 * is not accepted (of p, should that be 0 everywhere), or of p in row draft_len
 * where all are. Greedy: a proposal is accepted where it is the row's largest
 * logit's lowest index, which is also the next token; draft_probs do not enter.
 * Everything is computed in fp64 from the logits as given (exponentials to
 * 1.5e-14 of themselves). NaN and -inf logits have probability 0; where
 * logits are +inf, they share the row equally; a row with neither these nor
 * a finite logit accepts nothing and gives the token -1. A proposal outside
 * [0, V) is not accepted. Deterministic.
 *   workspace  moe_verify_draft_workspace_size() bytes; contents on entry do
 *              not matter and are clobbered
 * Two launches. Sizes: S >= 0 (S == 0 is a no-op), 1 <= W <=
 * K3MOE_MAX_VERIFY_WIDTH, 1 <= V <= K3MOE_MAX_VOCAB, and
 * S * W * ceil(V / 4096) < 2^24 (K3MOE_ERR_SHAPE). With W == 1 (plain sampling)
 * draft_ids, draft_probs, u_accept and accept_prob are not read or written and
 * may be NULL. Calls that overlap need workspaces of their own.
 */
size_t moe_verify_draft_workspace_size(int64_t S, int32_t W, int32_t V);
int moe_verify_draft(const void* logits, int32_t dtype, const int32_t* draft_ids, const float* draft_probs,
                     const int32_t* draft_len, const float* temperature, const float* u_accept, const float* u_sample,
                     int64_t S, int32_t W, int32_t V, int32_t* n_accepted, int32_t* tokens, float* accept_prob,
                     void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* K3MOE_SERVE_H */
