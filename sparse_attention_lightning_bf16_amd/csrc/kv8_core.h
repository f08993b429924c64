// Building blocks of the kernels that read the 8-bit cache: 16x16x32 matrix
// products of e4m3 keys and values against 16-bit queries and weights.
//
// Scores are computed transposed, keys as rows and queries as columns, so
// that a lane's column is one query for the scores, the softmax statistics
// and the output alike:
//   A (16 x 32): a[j] = A[l % 16][8 * (l / 16) + j]      j = 0..7
//   B (32 x 16): b[j] = B[8 * (l / 16) + j][l % 16]
//   C (16 x 16): c[i] = C[4 * (l / 16) + i][l % 16]      i = 0..3
// The order of the contraction index is free as long as both operands agree.
// For the scores a lane reads 16 consecutive codes of its key (dimensions
// 64 u + 16 g + 0..15, g = l / 16) and uses them in two steps.  For the output
// the scores of two 16-key tiles are already the B operand: a lane holds keys
// 16 (j / 4) + 4 g + j % 4 of its query as b[j], so it reads its values from
// those 8 keys: D / 16 consecutive codes of each, byte e of which belongs to
// output tile e, row l % 16.  No operand passes through LDS.
//
// Every e4m3 code is exact in bf16 and in fp16.
#pragma once

#include "common.h"
#include "launch_kv8.h"

namespace lix {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2v __attribute__((ext_vector_type(2)));

// The 16-bit types of queries: fragments, products, and two codes of a word
// (its lower or upper half) converted.
struct QBf16 {
    typedef __bf16 elem;
    typedef bf16x8 frag;
    // Attention weights are rounded to one fp16 (11 bits): below what an
    // output of 8 bits shows.
    static constexpr bool kTwoWeights = false;
    static __device__ __forceinline__ f32x4 mfma(const frag& a, const frag& b, const f32x4& c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    template <bool HI>
    static __device__ __forceinline__ uint32_t codes(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, HI));
    }
};
struct QFp16 {
    typedef _Float16 elem;
    typedef f16x8 frag;
    // An output of 11 bits would show one rounding of the weights to 11 bits
    // (1.48 times the error of its own rounding, measured): they are held as
    // the sum of two fp16, a second product with the remainder.
    static constexpr bool kTwoWeights = true;
    static __device__ __forceinline__ f32x4 mfma(const frag& a, const frag& b, const f32x4& c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    template <bool HI>
    static __device__ __forceinline__ uint32_t codes(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, HI));
    }
};

// Eight codes (two words) as one A fragment.
template <class Q>
__device__ __forceinline__ typename Q::frag key_frag(uint32_t w0, uint32_t w1) {
    const u32x4 v = {Q::template codes<false>(w0), Q::template codes<true>(w0), Q::template codes<false>(w1),
                     Q::template codes<true>(w1)};
    return __builtin_bit_cast(typename Q::frag, v);
}

// Bytes 4 w .. 4 w + 3 of the eight keys' words v[0..7] as four fp16 A
// fragments, one per byte: two v_perm interleave the bytes of a pair of keys,
// the conversion takes a 16-bit half (two keys' codes of one dimension).
__device__ __forceinline__ void value_frags(const uint32_t (&v)[8], f16x8 (&f)[4]) {
    u32x4 o[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t lo = __builtin_amdgcn_perm(v[2 * p + 1], v[2 * p], 0x05010400u);
        const uint32_t hi = __builtin_amdgcn_perm(v[2 * p + 1], v[2 * p], 0x07030602u);
        o[0][p] = QFp16::codes<false>(lo);
        o[1][p] = QFp16::codes<true>(lo);
        o[2][p] = QFp16::codes<false>(hi);
        o[3][p] = QFp16::codes<true>(hi);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __builtin_bit_cast(f16x8, o[e]);
}

// Nonzero bits where a byte of w is one of e4m3's NaN codes (0x7f, 0xff).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// max over the four lanes that hold a column (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float column_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float column_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Tokens that query t of sequence b sees, of a sequence of `len` tokens.
__device__ __forceinline__ int visible_tokens(const QueryArgs& q, int b, int t, int len) {
    if (q.q_lens != nullptr && t >= q.q_lens[b]) return 0;
    if (q.q_start == nullptr) return len;
    const long seen = ((long)q.q_start[b] + t + 1) / q.ratio;
    return (int)max(0L, min((long)len, seen));
}

__device__ __forceinline__ int cached_len(const KV8Pages& c, int b) {
    return (int)min((long)max(c.lens[b], 0), (long)c.max_pages << c.page_shift);
}

}  // namespace lix
