/*
 * k3moe_ops.h — microscaled 4-bit quantisation and products, and the routed
 * layer for a few tokens: the second half of libk3moe's C ABI.  Every general
 * convention of k3moe.h holds here too (device pointers, 16-byte alignment,
 * caller-owned buffers, host checks before anything is enqueued, status codes,
 * outputs fully overwritten, reentrancy).
 *
 * A microscaled 4-bit matrix [R, K] (K a multiple of 32) is a pair
 *   packed u8 [R, K/2]   E2M1 codes; element 2i of a row in the low nibble of
 *                        byte i, element 2i+1 in the high nibble
 *   scale  u8 [R, K/32]  E8M0 byte e of each 32 elements: the value 2^(e-127),
 *                        255 = NaN
 * (the compressed-tensors layout that mxfp4_repack reads).
 */
#ifndef K3MOE_OPS_H
#define K3MOE_OPS_H

#include "k3moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Input dtype beside K3MOE_DTYPE_F32 and K3MOE_DTYPE_BF16. */
#define K3MOE_DTYPE_F16 2
/* Largest K of the calls below. */
#define K3MOE_MAX_K_MX (1 << 20)

/*
 * mxfp4_quantize — float rows to microscaled 4 bits.
 * Source of the layout: llama.cpp pull request "model: add Kimi-K3 text
 * model", review comment "repack_mxfp4_blocks is bit-exact" (packed and scale
 * of one tensor).  The pages only read quantised weights; the rounding is the
 * OCP Microscaling Formats specification 1.0.
 *
 *   x       [R, K] f32, bf16 or f16 (x_dtype)
 *   packed  u8 [R, K/2], scale u8 [R, K/32]: out
 *
 * Block scale 2^e with e = max(floor(log2 m) - 2, -127), m = the block's
 * largest magnitude; with saturate == 0, e is one larger where m > 6 * 2^e, so
 * that no element is clamped.  A code is the E2M1 value nearest to v / 2^e,
 * ties to the even code, magnitudes above 6 clamped to 6, the sign kept (also
 * of zeros).  An all-zero block has scale byte 0.  A block holding an infinity
 * or a NaN gets scale byte 255 and the code 7 for every element: its values
 * read as NaN (mxfp4_unpack, mxfp4_matmul) or, through the 17-byte blocks of
 * mxfp4_repack, as +inf.
 * Sizes: R >= 0 (R == 0 is a no-op), 0 < K <= K3MOE_MAX_K_MX, K % 32 == 0,
 * R * K < 2^46 (K3MOE_ERR_SHAPE). Unknown x_dtype: K3MOE_ERR_UNSUPPORTED.
 */
int mxfp4_quantize(const void* x, int32_t x_dtype, int64_t R, int64_t K, int32_t saturate, uint8_t* packed,
                   uint8_t* scale, void* stream);

/*
 * mxfp4_unpack — the values of a microscaled matrix in the layout above:
 * out [R, K] f32 or bf16 (out_dtype), code * 2^(e-127), the sign of zero kept,
 * NaN for scale byte 255; exact, except that values beyond the largest finite
 * number (e = 254) become infinite. mxfp4_dequant is the same for 17-byte
 * blocks. Sizes and statuses as mxfp4_quantize.
 */
int mxfp4_unpack(const uint8_t* packed, const uint8_t* scale, int64_t R, int64_t K, int32_t out_dtype, void* out,
                 void* stream);

/*
 * mxfp4_matmul — product of two microscaled matrices,
 *   out[m][n] = sum_k A[m][k] * W[n][k],
 *   a_packed u8 [M, K/2], a_scale u8 [M, K/32]
 *   w_packed u8 [N, K/2], w_scale u8 [N, K/32]
 *   out [M, N] f32 or bf16 (out_dtype)
 * Exact products of the stored values, summed in fp32 on the block-scaled
 * matrix instructions, rounded once for a bf16 output. A row of A or W with a
 * NaN scale makes its row or column of out NaN. Deterministic.
 * Sizes: M >= 0 and N >= 0 (0: a no-op) up to 2^31 - 1, K as above;
 * K3MOE_ERR_SHAPE where M * N needs more than 2^31 - 1 tiles of 64 x 64.
 */
int mxfp4_matmul(const uint8_t* a_packed, const uint8_t* a_scale, const uint8_t* w_packed, const uint8_t* w_scale,
                 int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* out, void* stream);

/*
 * mxfp4_linear — float rows times a microscaled weight matrix: the rows are
 * quantised as mxfp4_quantize does (x_dtype, saturate) and multiplied as
 * mxfp4_matmul does, with the same bits as the two calls. Up to 16 rows of
 * together at most 32768 elements take one launch (the kernel quantises its
 * rows itself); more are quantised into the workspace first.
 *   workspace  mxfp4_linear_workspace_size() bytes (0: may be NULL); contents
 *              on entry do not matter and are clobbered
 */
size_t mxfp4_linear_workspace_size(int64_t M, int64_t N, int64_t K);
int mxfp4_linear(const void* x, int32_t x_dtype, const uint8_t* w_packed, const uint8_t* w_scale, int64_t M, int64_t N,
                 int64_t K, int32_t saturate, int32_t out_dtype, void* out, void* workspace, size_t workspace_bytes,
                 void* stream);

/* Most tokens of moe_mxfp4_layer. */
#define K3MOE_MAX_LAYER_TOKENS 16

/*
 * moe_mxfp4_layer — the routed layer of a few tokens in two launches: routing
 * as moe_route_topk, then the experts and their weighted sum as moe_mxfp4_ffn.
 * Sources: as those two (llama.cpp pull request "model: add Kimi-K3 text
 * model": expert count, used experts, sigmoid gating, exp_probs_b;
 * build_moe_ffn: route -> per-expert products -> weighted sum).
 *
 *   x_bf16   bf16 [T, D]         latent activations
 *   logits   f32 [T, E], bias f32 [E] or NULL, normalize, route_scale: routing
 *   w1, w3   u8 [E, I, D/32, 17], w2 u8 [E, D, I/32, 17]: expert matrices in
 *            the stage-tiled order of mxfp4_tile, as moe_mxfp4_ffn reads them
 *   out      f32 [T, D]
 *   topk_ids i32 [T, k], topk_w f32 [T, k]: optional outputs of the routing
 *            (NULL: kept in the workspace), the bits of moe_route_topk
 *   workspace  moe_mxfp4_layer_workspace_size() bytes; contents on entry do
 *            not matter and are clobbered
 *
 * Precision: exact weights, fp32 accumulation. x and h = SiLU(g) * u (fp32) enter
 * the products in fixed point per 32-element block, to 2^-24 of the block's
 * largest magnitude (elements of x down to 2^-17 of it exactly; blocks below
 * 2^-104 to 2^-128). The k expert outputs are summed in fp32 in slot order
 * (deterministic, no atomics on values). moe_mxfp4_ffn rounds h to about 16 bits,
 * so the two agree to that. A token with an infinite or NaN element of x, or with
 * an h beyond fp32, gets NaN outputs, as from moe_mxfp4_ffn, and no other token
 * does. The weights' E8M0 bytes must be <= 254. More than 1024 experts take a
 * third launch (the router's own).
 * An expert's weights are streamed once per two of its tokens, so tokens that
 * mostly choose different experts gain; where many share one, moe_route_topk and
 * moe_mxfp4_ffn stream less.
 * Sizes: 0 <= T <= K3MOE_MAX_LAYER_TOKENS (T == 0 is a no-op), D, I, E and k
 * as for moe_mxfp4_ffn. Calls that overlap (two streams, two graphs) need
 * workspaces of their own.
 */
size_t moe_mxfp4_layer_workspace_size(int64_t T, int32_t D, int32_t I, int32_t E, int32_t k);
int moe_mxfp4_layer(const void* x_bf16, const float* logits, const float* bias, const uint8_t* w1, const uint8_t* w3,
                    const uint8_t* w2, int64_t T, int32_t D, int32_t I, int32_t E, int32_t k, int32_t normalize,
                    float route_scale, int32_t act, float* out, int32_t* topk_ids, float* topk_w, void* workspace,
                    size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* K3MOE_OPS_H */
