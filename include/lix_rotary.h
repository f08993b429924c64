/*
 * lix_rotary.h - C ABI of liblix.so, rotary positions of queries and keys.
 *
 * The indexer takes queries and keys with their positions already in them
 * (page "nemo_automodel.components.models.deepseek_v41.indexer", section
 * indexer_scores: rotary embedding is applied before the call).  This entry
 * point applies them, and its inverse is the gradient.  The conventions of
 * lix.h hold (device memory of the current device, caller-owned, work on the
 * caller's stream, synchronous validation, its status codes), except that x
 * and out may be strided.
 */
#ifndef LIX_ROTARY_H
#define LIX_ROTARY_H

#include "lix.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the entry points that take more than one. */
typedef enum { LIX_BF16 = 0, LIX_FP16 = 1, LIX_FP32 = 2 } lix_dtype;

/* Which dimensions of the rotary part form a pair: (i, i + rot/2) or (2i, 2i+1). */
typedef enum { LIX_ROTARY_HALF = 0, LIX_ROTARY_INTERLEAVED = 1 } lix_rotary_layout;

/*
 * lix_rotary - rotates the pairs of a part of each head by its position.
 *
 * For token (i, j), head h and pair p = (a, b) of the dimensions
 * [start, start + rot), with angle = positions[i,j] * inv_freq[p]:
 *     out[a] = scale * (x[a] cos(angle) - x[b] sin(angle))
 *     out[b] = scale * (x[b] cos(angle) + x[a] sin(angle))
 * The other dimensions are copied unchanged.  inverse != 0 takes the negative
 * angle: with the same scale that is the gradient of x for the gradient of
 * out.  The angle is formed and reduced in 64 bits (a position of 10^6 times
 * an inverse frequency of 1 keeps 2^-30 of a turn), products and sums in 32,
 * rounded once to the type of out.
 *
 *   x          dtype [N0, N1, H, D], strides x_s0, x_s1, x_sh in elements,
 *              the last dimension contiguous
 *   positions  int32 [N0, N1], strides p_s0, p_s1 (0 broadcasts); any value
 *   inv_freq   fp64 [rot / 2]
 *   out        dtype [N0, N1, H, D] with its own strides; may be x itself
 *              with x's strides, may not overlap it otherwise
 * LIX_ERR_SHAPE: a size < 1, rot odd or < 2, start < 0 or start + rot > D, a
 * layout or dtype that is not listed, or a negative stride.
 * LIX_ERR_UNSUPPORTED: D > 1024, or a pointer not aligned to its element.
 */
int lix_rotary(const void* x, long long x_s0, long long x_s1, long long x_sh,
               const int32_t* positions, long long p_s0, long long p_s1, const double* inv_freq,
               int N0, int N1, int H, int D, int rot, int start, int layout, float scale, int inverse, int dtype,
               void* out, long long o_s0, long long o_s1, long long o_sh, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIX_ROTARY_H */
