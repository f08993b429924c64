// The attention weight that each cached token got (lix_kv8_token_weights):
//     w[s] = sum over the rows (queries x heads of a key head) that see s of
//            2^(scale log2(e) k_scale (q . code[s]) - log2(e) lse)
//
// A wave owns 16 KT keys of one key head: their codes are converted once to
// operand fragments that stay in registers, and the rows pass by, 16 at a
// time.  Keys are the rows of the product (kv8_core.h), so a lane adds up its
// own keys over all rows it sees and the sum over the 16 row columns is taken
// once at the end: no atomics, the same order on every call.  One query: bound
// by reading the key codes; many: by the exponentials.
#include <hip/hip_runtime.h>

#include "kv8_core.h"

namespace lix {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

template <class Q, int D, int KT>
__global__ __launch_bounds__(256, 2) void kv8_weights_kernel(WeighArgs a) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long pairs = (long)a.q.B * a.c.Hkv;
    const long pair = blockIdx.x % pairs;
    const int b = (int)(pair / a.c.Hkv), kvh = (int)(pair % a.c.Hkv);
    const int len = cached_len(a.c, b);
    const long s_first = (blockIdx.x / pairs * 4 + wave) * (16L * KT);
    if (s_first >= len) return;
    const int s0 = (int)s_first;
    const int shift = a.c.page_shift;

    typename Q::frag key[KT][D / 32];
    float c[KT];
    bool exists[KT];
#pragma unroll
    for (int h = 0; h < KT; ++h) {
        const int s = s0 + 16 * h;
        const int nth = s >> shift;
        int pid = nth < a.c.max_pages ? a.c.table[(long)b * a.c.max_pages + nth] : -1;
        exists[h] = s < len && pid >= 0 && pid < a.c.num_pages;
        pid = exists[h] ? pid : 0;
        const long at = (long)pid * a.c.Hkv + kvh;
        const uint8_t* p = a.c.k + ((at << shift) + (s & ((1 << shift) - 1)) + (lane & 15)) * D + 16 * g;
        c[h] = exists[h] ? a.c.k_scale[at] * a.q.scale_log2 : 0.0f;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(p + 64 * u);
            key[h][2 * u] = key_frag<Q>(w[0], w[1]);
            key[h][2 * u + 1] = key_frag<Q>(w[2], w[3]);
        }
    }

    f32x4 sum[KT];
#pragma unroll
    for (int h = 0; h < KT; ++h) sum[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const typename Q::elem* q = static_cast<const typename Q::elem*>(a.q.q) + b * a.q.sb + 16 * g;
    const int rows = a.q.S * a.q.G;
    // rows before the first query that sees this wave's first key add nothing
    int first = 0;
    if (a.q.q_start != nullptr) {
        const long t = ((long)s0 + 1) * a.q.ratio - 1 - a.q.q_start[b];
        first = (int)min(max(t, 0L), (long)a.q.S) * a.q.G;
    }
    for (int r0 = first; r0 < rows; r0 += 16) {
        const int r = min(r0 + (lane & 15), rows - 1);
        const int t = r / a.q.G, head = kvh * a.q.G + r - t * a.q.G;
        typename Q::frag f[D / 32];
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks)
            f[ks] = *reinterpret_cast<const typename Q::frag*>(q + t * a.q.ss + head * a.q.sh + 64 * (ks / 2) +
                                                               8 * (ks & 1));
        const float lse = a.lse[((long)b * a.q.S + t) * a.q.Hq + head];
        int vis = r0 + (lane & 15) < rows ? visible_tokens(a.q, b, t, len) : 0;
        if (lse == neg_inf()) vis = 0;
        const float base = -lse * kLog2e;
        const bool edge = __any(vis < s0 + 16 * KT) || s0 + 16 * KT > len;
#pragma unroll
        for (int h = 0; h < KT; ++h) {
            f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) x = Q::mfma(key[h][ks], f[ks], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float p = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], c[h], base));
                if (edge) p = s0 + 16 * h + 4 * g + i < vis ? p : 0.0f;
                sum[h][i] += p;
            }
        }
    }
    // over the 16 columns; lane l % 16 == i writes key 4 g + i
#pragma unroll
    for (int h = 0; h < KT; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = sum[h][i];
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) v += __shfl_xor(v, o);
            const int s = s0 + 16 * h + 4 * g + i;
            if ((lane & 15) == i && s < len) {
                float* w = a.weights + pair * a.width + s;
                const float got = exists[h] ? v : 0.0f;
                *w = a.accumulate ? *w + got : got;
            }
        }
}

template <class Q, int D>
hipError_t launch(const WeighArgs& a) {
    const long cap = (long)a.c.max_pages << a.c.page_shift;
    const long pairs = (long)a.q.B * a.c.Hkv;
    // 64 keys a wave read each row of queries least often; with one row tile
    // there is nothing to share, and 32 keys a wave spread further
    auto go = [&](auto kernel, long keys) {
        const long grid = pairs * ((cap + 4 * keys - 1) / (4 * keys));
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, a.stream, a);
    };
    if (a.q.S * a.q.G > 16 && D <= 128) go(kv8_weights_kernel<Q, D, 4>, 64);
    else go(kv8_weights_kernel<Q, D, 2>, 32);
    return hipGetLastError();
}

template <class Q>
hipError_t launch_dim(const WeighArgs& a) {
    switch (a.c.D) {
        case 64: return launch<Q, 64>(a);
        case 128: return launch<Q, 128>(a);
        default: return launch<Q, 256>(a);
    }
}

}  // namespace

hipError_t launch_kv8_token_weights(const WeighArgs& a) {
    return a.q.dtype == LIX_BF16 ? launch_dim<QBf16>(a) : launch_dim<QFp16>(a);
}

}  // namespace lix
