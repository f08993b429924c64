// Filling the 8-bit cache (lix_kv8_append) and cutting it to its heaviest
// tokens (lix_kv8_evict).
//
// Both write pages of e4m3 codes with one scale per page and head.  A
// workgroup owns one (page, head) of the keys or of the values: it holds the
// page's new values in registers (8 of a row per piece), takes their largest
// magnitude over the workgroup, and writes the codes and the scale, so every
// value is read once and no two workgroups write the same bytes.  Bound by
// memory for prompts, by latency for single tokens.
#include <hip/hip_runtime.h>

#include "kv8_quant.h"
#include "launch.h"
#include "launch_kv8.h"

namespace lix {

namespace {

constexpr int kThreads = 256;

// Eight 16-bit floats of type T as fp32.
template <class T>
__device__ __forceinline__ void unpack8(const u32x4& w, float (&x)[8]) {
    typedef T t8 __attribute__((ext_vector_type(8)));
    const t8 v = __builtin_bit_cast(t8, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}

// ---------------------------------------------------------------- append

// One workgroup per (sequence, head, keys or values, j-th page that the new
// tokens may fall on).  CH: pieces of 8 values a thread holds at most.
template <class T, int CH>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(AppendArgs a, int pages) {
    __shared__ float part[4];
    const int j = blockIdx.x % pages;
    int rest = blockIdx.x / pages;
    const int which = rest & 1;
    rest >>= 1;
    const int h = rest % a.c.Hkv, b = rest / a.c.Hkv;
    const int shift = a.c.page_shift, D = a.c.D;

    const long cap = (long)a.c.max_pages << shift;
    const long len = min((long)max(a.c.lens[b], 0), cap);
    const int fresh = a.new_lens ? min(max(a.new_lens[b], 0), a.S) : a.S;
    const long nth = (len >> shift) + j;
    const long lo = max(len, nth << shift), hi = min(len + fresh, (nth + 1) << shift);
    if (lo >= hi || nth >= a.c.max_pages) return;
    const int pid = a.c.table[(long)b * a.c.max_pages + nth];
    if (pid < 0 || pid >= a.c.num_pages) return;

    const int per_row = D >> 3;                       // pieces of a row
    const int n = (int)(hi - lo) * per_row;
    const int first = (int)(lo - (nth << shift));     // first new slot of the page
    // two selects and no run-time index: a kernel argument array indexed at
    // run time would be copied to scratch
    const T* x = static_cast<const T*>(which ? a.x[1] : a.x[0]);
    const long sb = which ? a.sb[1] : a.sb[0], ss = which ? a.ss[1] : a.ss[0], sh = which ? a.sh[1] : a.sh[0];
    x += b * sb + (lo - len) * ss + h * sh;

    u32x4 raw[CH];
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * kThreads + threadIdx.x;
        raw[c] = u32x4{0, 0, 0, 0};
        if (i < n) {
            const int row = i / per_row, p = i - row * per_row;
            raw[c] = *reinterpret_cast<const u32x4*>(x + row * ss + p * 8);
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        float f[8];
        unpack8<T>(raw[c], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = finite_top(top, f[e]);
    }
    top = workgroup_max(top, part);

    const long at = (long)pid * a.c.Hkv + h;
    float* scale_at = (which ? a.c.v_scale : a.c.k_scale) + at;
    uint8_t* codes = (which ? a.c.v : a.c.k) + ((at * D) << shift);
    float scale = page_scale(top);
    if (first > 0) {
        const float before = *scale_at;
        scale = fmaxf(before, scale);
        if (scale != before) {                        // older tokens at the larger scale
            for (int i = threadIdx.x; i < first * D / 4; i += kThreads) {
                float f[4];
                uint32_t* w = reinterpret_cast<uint32_t*>(codes) + i;
                e4m3_quad_to_f32(*w, f);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] *= before;
                *w = e4m3_quad(f, scale);
            }
        }
        __syncthreads();                              // every thread has read the old scale
    }
    if (threadIdx.x == 0) *scale_at = scale;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * kThreads + threadIdx.x;
        if (i < n) {
            float f[8];
            unpack8<T>(raw[c], f);
            const float lo4[4] = {f[0], f[1], f[2], f[3]}, hi4[4] = {f[4], f[5], f[6], f[7]};
            const uint2 w = make_uint2(e4m3_quad(lo4, scale), e4m3_quad(hi4, scale));
            *reinterpret_cast<uint2*>(codes + (long)first * D + i * 8) = w;
        }
    }
}

template <class T>
hipError_t launch_append(const AppendArgs& p) {
    const int page = 1 << p.c.page_shift;
    const int pages = (p.S + page - 1) / page + 1;    // S tokens, starting anywhere in a page
    const long grid = (long)p.B * p.c.Hkv * 2 * pages;
    const int pieces = (p.S < page ? p.S : page) * p.c.D / 8;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kThreads), 0, p.stream, p, pages);
    };
    if (pieces <= kThreads) go(kv8_append_kernel<T, 1>);
    else if (pieces <= 4 * kThreads) go(kv8_append_kernel<T, 4>);
    else go(kv8_append_kernel<T, 16>);
    return hipGetLastError();
}

// ---------------------------------------------------------------- evict

// Tokens kept of a sequence of n: all if n <= keep, else the first `sinks`,
// `middle` selected ones in ascending order, and the last `recent`.
__device__ __forceinline__ int kept_token(const EvictArgs& a, const int32_t* __restrict__ mid, int middle, int n, int j) {
    if (n <= a.keep || j < a.sinks) return j;
    return j < a.sinks + middle ? mid[j - a.sinks] : n - a.keep + j;
}

__device__ __forceinline__ int evict_len(const EvictArgs& a, int b) {
    return (int)min((long)max(a.c.lens[b], 0), (long)a.c.max_pages << a.c.page_shift);
}

// Range of the tokens that compete by weight, per (sequence, head) row.
__global__ __launch_bounds__(kThreads) void kv8_evict_ranges_kernel(EvictArgs a, int32_t* begin, int32_t* end) {
    const int row = blockIdx.x * kThreads + threadIdx.x;
    if (row >= a.B * a.c.Hkv) return;
    const int n = evict_len(a, row / a.c.Hkv);
    begin[row] = a.sinks;
    end[row] = n <= a.keep ? a.sinks : n - a.recent;
}

// One workgroup per (sequence, head, keys or values, new page): the kept rows
// are read once into registers, as codes with the scale of their old page.
template <int CH>
__global__ __launch_bounds__(kThreads) void kv8_evict_kernel(EvictArgs a, const int32_t* __restrict__ indices, int middle,
                                                              int pages) {
    __shared__ float part[4];
    const int j = blockIdx.x % pages;
    int rest = blockIdx.x / pages;
    const int which = rest & 1;
    const int row = rest >> 1;
    const int h = row % a.c.Hkv, b = row / a.c.Hkv;
    const int shift = a.c.page_shift, page = 1 << shift, D = a.c.D;
    const int n = evict_len(a, b);
    const int count = min(n, a.keep);
    const int32_t* mid = indices + (long)row * middle;
    if (which == 0) {
        if (h == 0 && j == 0 && threadIdx.x == 0) a.new_lens[b] = count;
        const int slot = (j << shift) + threadIdx.x;
        if (threadIdx.x < page && slot < a.keep) {
            const int s = slot < count ? kept_token(a, mid, middle, n, slot) : -1;
            a.kept[(long)row * a.keep + slot] = s;
            a.new_weights[(long)row * a.keep + slot] = s < 0 ? 0.0f : a.weights[(long)row * a.width + s];
        }
    }
    const int first = j << shift;
    if (first >= count) return;
    const int pid = a.new_table[(long)b * a.new_max_pages + j];
    if (pid < 0 || pid >= a.c.num_pages) return;

    const uint8_t* src = which ? a.c.v : a.c.k;
    const float* src_scale = which ? a.c.v_scale : a.c.k_scale;
    const int per_row = D >> 4;                       // pieces of 16 codes
    const int pieces = min(page, count - first) * per_row;
    u32x4 raw[CH];
    float scales[CH];
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * kThreads + threadIdx.x;
        raw[c] = u32x4{0, 0, 0, 0};
        scales[c] = 0.0f;
        if (i < pieces) {
            const int r = i / per_row, p = i - r * per_row;
            const int s = kept_token(a, mid, middle, n, first + r);
            const int old = s < 0 ? -1 : a.c.table[(long)b * a.c.max_pages + (s >> shift)];
            if (old >= 0 && old < a.c.num_pages) {
                const long at = (long)old * a.c.Hkv + h;
                raw[c] = *reinterpret_cast<const u32x4*>(src + ((at << shift) + (s & (page - 1))) * D + p * 16);
                scales[c] = src_scale[at];
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float f[4];
            e4m3_quad_to_f32(raw[c][w], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) top = finite_top(top, f[e] * scales[c]);
        }
    top = workgroup_max(top, part);
    const float scale = page_scale(top);
    const long at = (long)pid * a.c.Hkv + h;
    if (threadIdx.x == 0) (which ? a.c.v_scale : a.c.k_scale)[at] = scale;
    uint8_t* codes = (which ? a.c.v : a.c.k) + ((at * D) << shift);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * kThreads + threadIdx.x;
        if (i < pieces) {
            u32x4 o;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float f[4];
                e4m3_quad_to_f32(raw[c][w], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] *= scales[c];
                o[w] = e4m3_quad(f, scale);
            }
            *reinterpret_cast<u32x4*>(codes + (long)i * 16) = o;
        }
    }
}

}  // namespace

hipError_t launch_kv8_append(const AppendArgs& p) {
    return p.dtype == LIX_BF16 ? launch_append<__bf16>(p) : launch_append<_Float16>(p);
}

// The middle tokens are selected by the row top-k of the indexer, one row per
// (sequence, head), over the range that competes; a row that keeps all has an
// empty one.
hipError_t launch_kv8_evict(const EvictArgs& p, const EvictLayout& ly) {
    char* ws = static_cast<char*>(p.workspace);
    int32_t* indices = reinterpret_cast<int32_t*>(ws + ly.indices);
    const int rows = p.B * p.c.Hkv;
    if (ly.middle > 0) {
        int32_t* begin = reinterpret_cast<int32_t*>(ws + ly.begin);
        int32_t* end = reinterpret_cast<int32_t*>(ws + ly.end);
        hipLaunchKernelGGL(kv8_evict_ranges_kernel, dim3((rows + kThreads - 1) / kThreads), dim3(kThreads), 0, p.stream,
                           p, begin, end);
        TopkArgs t{p.weights, 1, rows, p.width, 1, ly.middle, begin, end, reinterpret_cast<float*>(ws + ly.scores),
                   indices, p.stream};
        const hipError_t e = launch_topk_rows(t);
        if (e != hipSuccess) return e;
    }
    const int page = 1 << p.c.page_shift;
    const int pages = (p.keep + page - 1) / page;
    const long grid = (long)rows * 2 * pages;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kThreads), 0, p.stream, p, indices, ly.middle, pages);
    };
    const int pieces = page * p.c.D / 16;
    if (pieces <= kThreads) go(kv8_evict_kernel<1>);
    else if (pieces <= 2 * kThreads) go(kv8_evict_kernel<2>);
    else go(kv8_evict_kernel<8>);
    return hipGetLastError();
}

}  // namespace lix
