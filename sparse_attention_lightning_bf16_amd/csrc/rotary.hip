// Rotary positions: each pair (a, b) of the rotary part of a head is turned
// by angle = position * inv_freq[pair]:
//     out_a = scale (a cos - b sin),  out_b = scale (b cos + a sin)
// and the rest of the head is copied.  The inverse turn is the gradient.
//
// Bound by memory: one read and one write of every element.  The angles of a
// token serve all its heads, so a workgroup takes whole tokens: its threads
// first put the cosines and sines of its tokens into LDS (rot / 2 each), then
// stream the tokens' heads in 16-byte pieces.  A workgroup takes as many
// tokens as make four pieces a thread, so that short tokens (one key head)
// still fill it.
//
// The angle is position * inv_freq / (2 pi) turns in fp64, reduced there to
// [-1/2, 1/2] and only then rounded to fp32: a far position keeps its angle.
#include <hip/hip_runtime.h>

#include "common.h"
#include "launch_kv8.h"

namespace lix {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;        // cosines and sines of a workgroup's tokens in LDS

template <class T>
__device__ __forceinline__ float to_f32(T x) { return (float)x; }
template <class T>
__device__ __forceinline__ T from_f32(float x) { return (T)x; }

// VEC elements of one thread: 16 bytes where everything is a multiple of
// that, one element otherwise.
template <class T, int VEC>
struct alignas(sizeof(T) * VEC) Piece {
    T v[VEC];
};

// Work of a token, in pieces of VEC elements:
//   interleaved: D / VEC pieces, a piece of the rotary part holds VEC / 2 pairs
//   half: a piece of the first half of the rotary part is taken together with
//         its partner in the second, so D / VEC - rot / (2 VEC) items
// With VEC = 1 an interleaved item is one pair or one copied element.
template <class T, int VEC, bool HALF>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, int tokens_per_wg, int items, int copied) {
    extern __shared__ float2 turn[];              // [tokens_per_wg][rot / 2]: scale cos, scale sin
    const int pairs = a.rot / 2;
    const long first = (long)blockIdx.x * tokens_per_wg;
    const long tokens = (long)a.N0 * a.N1;
    const int here = (int)min((long)tokens_per_wg, tokens - first);
    for (int i = threadIdx.x; i < here * pairs; i += kThreads) {
        const int tok = i / pairs;
        const long t = first + tok;
        const int n0 = (int)(t / a.N1), n1 = (int)(t - (long)n0 * a.N1);
        const double at = (double)a.positions[n0 * a.p_s0 + n1 * a.p_s1] * a.inv_freq[i - tok * pairs] *
                          0.15915494309189533577;
        float s, c;
        sincospif(2.0f * (float)(at - rint(at)), &s, &c);
        turn[i] = make_float2(a.scale * c, a.inverse ? -a.scale * s : a.scale * s);
    }
    __syncthreads();
    const T* __restrict__ x = static_cast<const T*>(a.x);
    T* __restrict__ out = static_cast<T*>(a.out);
    const int per_token = a.H * items;
    const int turned = items - copied;
    using P = Piece<T, VEC>;
    for (int i = threadIdx.x; i < here * per_token; i += kThreads) {
        const int tok = i / per_token;
        const int r = i - tok * per_token;
        const int h = r / items, it = r - h * items;
        const long t = first + tok;
        const int n0 = (int)(t / a.N1), n1 = (int)(t - (long)n0 * a.N1);
        const T* xs = x + n0 * a.x_s0 + n1 * a.x_s1 + h * a.x_sh;
        T* os = out + n0 * a.o_s0 + n1 * a.o_s1 + h * a.o_sh;
        if (it >= turned) {                       // copied: before and behind the rotary part
            int d = (it - turned) * VEC;
            if (d >= a.start) d += a.rot;
            *reinterpret_cast<P*>(os + d) = *reinterpret_cast<const P*>(xs + d);
            continue;
        }
        const float2* cs = turn + tok * pairs;
        if constexpr (HALF) {
            const int p0 = it * VEC, d = a.start + p0;
            const P u = *reinterpret_cast<const P*>(xs + d);
            const P w = *reinterpret_cast<const P*>(xs + d + pairs);
            P ou, ow;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 f = cs[p0 + e];
                const float ua = to_f32(u.v[e]), wb = to_f32(w.v[e]);
                ou.v[e] = from_f32<T>(ua * f.x - wb * f.y);
                ow.v[e] = from_f32<T>(wb * f.x + ua * f.y);
            }
            *reinterpret_cast<P*>(os + d) = ou;
            *reinterpret_cast<P*>(os + d + pairs) = ow;
        } else if constexpr (VEC == 1) {
            const int d = a.start + 2 * it;
            const float2 f = cs[it];
            const float ua = to_f32(xs[d]), wb = to_f32(xs[d + 1]);
            os[d] = from_f32<T>(ua * f.x - wb * f.y);
            os[d + 1] = from_f32<T>(wb * f.x + ua * f.y);
        } else {
            const int d = a.start + it * VEC;
            const P u = *reinterpret_cast<const P*>(xs + d);
            P o;
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                const float2 f = cs[it * (VEC / 2) + e / 2];
                const float ua = to_f32(u.v[e]), wb = to_f32(u.v[e + 1]);
                o.v[e] = from_f32<T>(ua * f.x - wb * f.y);
                o.v[e + 1] = from_f32<T>(wb * f.x + ua * f.y);
            }
            *reinterpret_cast<P*>(os + d) = o;
        }
    }
}

template <class T, int VEC>
hipError_t launch(const RotaryArgs& p) {
    const bool half = p.layout == LIX_ROTARY_HALF;
    const int copied = (p.D - p.rot) / VEC;
    const int items = copied + (half ? p.rot / (2 * VEC) : VEC == 1 ? p.rot / 2 : p.rot / VEC);
    const int pairs = p.rot / 2;
    const long tokens = (long)p.N0 * p.N1;
    int per_wg = max(1, 4 * kThreads / (p.H * items));
    per_wg = (int)min((long)max(1, min(per_wg, kMaxPairs / pairs)), tokens);
    const dim3 grid((unsigned)((tokens + per_wg - 1) / per_wg));
    const size_t lds = (size_t)per_wg * pairs * sizeof(float2);
    if (half)
        hipLaunchKernelGGL((rotary_kernel<T, VEC, true>), grid, dim3(kThreads), lds, p.stream, p, per_wg, items,
                           copied);
    else
        hipLaunchKernelGGL((rotary_kernel<T, VEC, false>), grid, dim3(kThreads), lds, p.stream, p, per_wg, items,
                           copied);
    return hipGetLastError();
}

template <class T>
hipError_t launch_type(const RotaryArgs& p) {
    constexpr int VEC = 16 / (int)sizeof(T);
    // a size-one dimension's stride reaches no address
    auto whole = [&](long s0, long s1, long sh) {
        return (p.N0 == 1 || s0 % VEC == 0) && (p.N1 == 1 || s1 % VEC == 0) && (p.H == 1 || sh % VEC == 0);
    };
    const bool vec = p.D % VEC == 0 && p.start % VEC == 0 &&
                     p.rot % (p.layout == LIX_ROTARY_HALF ? 2 * VEC : VEC) == 0 && whole(p.x_s0, p.x_s1, p.x_sh) &&
                     whole(p.o_s0, p.o_s1, p.o_sh) && ((uintptr_t)p.x | (uintptr_t)p.out) % 16 == 0;
    return vec ? launch<T, VEC>(p) : launch<T, 1>(p);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& p) {
    switch (p.dtype) {
        case LIX_BF16: return launch_type<__bf16>(p);
        case LIX_FP16: return launch_type<_Float16>(p);
        default: return launch_type<float>(p);
    }
}

}  // namespace lix
