/*
 * moe.h -- C ABI of a routed gated MLP ("mixture of experts") with 4-bit
 * block-quantized experts, for a few tokens.
 *
 * For each token t with router logits l [E]:
 *   the top_k experts of the largest logits (the lower index at ties), with
 *     weight softmax(l)_e, divided by the sum of the chosen ones if renormalize
 *   g = W1_e x,  u = W3_e x,  h = g / (1 + exp(-g)) * u          (float32)
 *   y = sum over the chosen e, in order of falling logits, of weight_e * (W2_e h)
 * A logit that is -infinity or NaN takes its expert out; a token with fewer
 * than top_k experts left uses those, one with none gives zeros.
 *
 * The products are those of q4_gemv: x and h are quantized per block to int8
 * (q4_quantize_act), each block's dot is an exact integer, and the block's
 * scales (and the affine bias) are applied in float32. Unlike there, a block
 * with a NaN has a NaN scale: a token with a NaN or an infinity gives NaN.
 *
 * Layouts (codes, scales and formats of q4.h, bits = 4):
 *   w13 [E][2 I][H/2] codes: rows 0 .. I-1 of an expert are W1 (gate), rows I .. 2I-1 W3 (up);
 *   s13, b13 [E][2 I][H/bs];  w2 [E][H][I/2];  s2, b2 [E][H][I/bs]
 * Only the chosen experts' weights are read, W1 and W3 once for each 4 to 16 of
 * an expert's tokens (about twice the mean number of an expert, as far as their
 * codes fit a CU's LDS; 1 for very long rows), W2 once for each 8, or 16 on the
 * matrix cores.
 *
 * Conventions (pointers, streams, workspaces, statuses) are those of q4.h.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the workspace of moe_q4 (0 for sizes that it refuses). */
size_t moe_q4_work_bytes(int T, int H, int I, int E, int top_k, int bs);

/*
 * x [T][H] (xdtype Q4_DT_F32 or Q4_DT_BF16, 16-byte aligned), logits [T][E] float32, y [T][H] in xdtype, 16-byte
 * aligned. bs = 32 for Q4_FMT_Q4_0, 64 or 128 for Q4_FMT_AFFINE (b13, b2 only there). H and I are multiples of bs.
 * 1 <= T <= 64, 1 <= E <= 512, 1 <= top_k <= min(E, 16), H and I at most 32768, an expert's codes below 2^31 bytes.
 * work: moe_q4_work_bytes(...) bytes, 16-byte aligned. Two launches.
 */
int moe_q4(int T, int H, int I, int E, int top_k, int bs, int fmt, int xdtype, const void* x, const float* logits,
           const uint8_t* w13, const void* s13, const void* b13, const uint8_t* w2, const void* s2, const void* b2,
           int renormalize, void* y, void* work, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
