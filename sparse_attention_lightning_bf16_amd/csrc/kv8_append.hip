// Filling the 8-bit cache (lix_kv8_append) and cutting it to its heaviest
// tokens (lix_kv8_evict).
//
// Both write pages of e4m3 codes with one scale per page and head.  A
// workgroup owns a (page, head): it holds the
// page's new values in registers, takes their largest
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
    __shared__ float part[2][4];
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
        for (int e = 0; e < 8; e += 2) top = fmaxf(top, fmaxf(fabsf(f[e]), fabsf(f[e + 1])));     // NaN is passed over
    }
    top = workgroup_max(top, part[0]);
    // Rare: infinities, which do not count for the scale and saturate.
    const bool infinite = top == kInf;
    if (infinite) {
        top = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float f[8];
            unpack8<T>(raw[c], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = finite_top(top, f[e]);
        }
        top = workgroup_max(top, part[1]);
    }

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
                for (int e = 0; e < 4; ++e) f[e] = f[e] * before / scale;
                *w = e4m3_quad<true>(f);
            }
        }
        __syncthreads();                              // every thread has read the old scale
    }
    if (threadIdx.x == 0) *scale_at = scale;
    // A power of two, as every scale that this call gives: its reciprocal is
    // exact.  Another one, of a page with older tokens, takes a division.
    const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0 && scale >= 0x1p-120f && scale <= 0x1p120f;
    const float inv = exact ? 1.0f / scale : 1.0f, by = exact ? 1.0f : scale;
    auto write = [&](auto general) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = c * kThreads + threadIdx.x;
            if (i < n) {
                float f[8];
                unpack8<T>(raw[c], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = general ? f[e] / by * inv : f[e] * inv;
                const float lo4[4] = {f[0], f[1], f[2], f[3]}, hi4[4] = {f[4], f[5], f[6], f[7]};
                const uint2 w = make_uint2(e4m3_quad<general>(lo4), e4m3_quad<general>(hi4));
                *reinterpret_cast<uint2*>(codes + (long)first * D + i * 8) = w;
            }
        }
    };
    if (exact && !infinite) write(std::false_type{});
    else write(std::true_type{});
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

// Selection: one workgroup per (sequence, head) row, its weights in registers
// (NPT of each of 1024 threads, token 1024 i + thread).  The m-th largest of
// the competing weights is found among their order-preserving keys: a histogram
// of 2048 bins between the smallest and the largest gives its bin, and bisection
// the key within: a step counts the keys at or above the middle (compare, ballot,
// population count) and stops early where exactly m are.  The bin's keys are first
// dealt out to the threads, one or two to each, unless there are too many.  Equal keys at the border go to the lowest tokens.  Kept tokens are
// written in order through the counts before each wave's group of 64.
//
// Rows beyond 32768 tokens take the indexer's row top-k instead, which reads a
// row several times; that one needs thousands of rows to fill the card (57 us
// for 64 rows of 32768, this 18).
constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64, kBins = 2 * kSelThreads;

__device__ __forceinline__ int evict_len(const EvictArgs& a, int b) {
    return (int)min((long)max(a.c.lens[b], 0), (long)a.c.max_pages << a.c.page_shift);
}

template <int NPT>
__global__ __launch_bounds__(kSelThreads) void kv8_select_kernel(EvictArgs a) {
    __shared__ uint32_t bounds[2][kSelWaves];
    __shared__ int counts[2][kSelWaves];
    __shared__ int above[NPT * kSelWaves], equal[NPT * kSelWaves];
    __shared__ int bins[kBins], found[4];
    const int row = blockIdx.x, b = row / a.c.Hkv;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = evict_len(a, b);
    const int count = min(n, a.keep);
    int32_t* kept = a.kept + (long)row * a.keep;
    float* new_w = a.new_weights + (long)row * a.keep;
    const float* w = a.weights + (long)row * a.width;
    if (tid == 0 && row == b * a.c.Hkv) a.new_lens[b] = count;
    for (int j = count + tid; j < a.keep; j += kSelThreads) {
        kept[j] = -1;
        new_w[j] = 0.0f;
    }
    float v[NPT];
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        // unconditional loads: behind the sequence its last token again
        v[i] = w[min(i * kSelThreads + tid, max(n - 1, 0))];
    }
    if (n <= a.keep) {
#pragma unroll
        for (int i = 0; i < NPT; ++i) {
            const int s = i * kSelThreads + tid;
            if (s < n) {
                kept[s] = s;
                new_w[s] = v[i];
            }
        }
        return;
    }
    // keys: 0 behind the sequence, kEnd for the ends that are kept without competing
    constexpr uint32_t kEnd = ~0u;
    const int lo_end = a.sinks, hi_end = n - a.recent;
    const int ends = a.sinks + a.recent, m = a.keep - ends;
    uint32_t key[NPT], least = ~0u, most = 0;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        const int s = i * kSelThreads + tid;
        const bool in = s >= lo_end && s < hi_end;
        const uint32_t k = min(max(f32_to_key(v[i]), 1u), kEnd - 1);
        key[i] = in ? k : s < n ? kEnd : 0u;
        least = min(least, in ? k : ~0u);
        most = max(most, in ? k : 0u);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        least = min(least, (uint32_t)__shfl_xor((int)least, o));
        most = max(most, (uint32_t)__shfl_xor((int)most, o));
    }
    if (lane == 0) {
        bounds[0][wave] = least;
        bounds[1][wave] = most;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSelWaves; ++i) {
        least = min(least, bounds[0][i]);
        most = max(most, bounds[1][i]);
    }
    // The bin that holds the m-th largest key: `over` keys are in higher ones.
    int sh = 0;
    while ((most - least) >> sh >= kBins) ++sh;
    for (int i = tid; i < kBins; i += kSelThreads) bins[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NPT; ++i)
        if (key[i] >= least && key[i] <= most) atomicAdd(&bins[(key[i] - least) >> sh], 1);
    __syncthreads();
    // thread t has bins kBins - 2 - 2 t and the one above it, highest first
    const int b_hi = bins[kBins - 1 - 2 * tid], b_lo = bins[kBins - 2 - 2 * tid];
    int before_t = b_hi + b_lo;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(before_t, o);
        before_t += lane >= o ? x : 0;
    }
    if (lane == 63) counts[0][wave] = before_t;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSelWaves; ++i) before_t += i < wave ? counts[0][i] : 0;
    before_t -= b_hi + b_lo;           // keys in higher bins
    if (before_t < m && m <= before_t + b_hi + b_lo) {
        const bool high = m <= before_t + b_hi;
        found[0] = kBins - 2 - 2 * tid + (high ? 1 : 0);
        found[1] = before_t + (high ? 0 : b_hi);
        found[2] = high ? b_hi : b_lo;
        found[3] = 0;
    }
    __syncthreads();
    uint32_t lo = least, hi = most;
    int over = 0;
    if (m > 0) {
        lo = least + ((uint32_t)found[0] << sh);
        hi = min(most, lo + ((1u << sh) - 1));
        over = found[1];
        // few keys in the bin: one or two of them to a thread
        const bool few = found[2] <= 2 * kSelThreads;
        uint32_t own[2] = {0, 0};
        if (few) {
#pragma unroll
            for (int i = 0; i < NPT; ++i)
                if (key[i] >= lo && key[i] <= hi) bins[atomicAdd(&found[3], 1)] = (int)key[i];
            __syncthreads();
            own[0] = tid < found[2] ? (uint32_t)bins[tid] : 0u;
            own[1] = tid + kSelThreads < found[2] ? (uint32_t)bins[tid + kSelThreads] : 0u;
        }
        // invariant: at least m keys are >= lo, fewer than m are >= hi + 1
        int side = 0;
        bool exact = false;            // m keys are >= lo, and no more
        while (lo < hi && !exact) {
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            int c = 0;
            if (few) {
                c = over * (wave == 0) + __popcll(__ballot(own[0] >= mid)) + __popcll(__ballot(own[1] >= mid));
            } else {
#pragma unroll
                for (int i = 0; i < NPT; ++i) c += __popcll(__ballot(key[i] >= mid));
                c -= wave == 0 ? ends : 0;
            }
            if (lane == 0) counts[side][wave] = c;
            __syncthreads();
            c = 0;
#pragma unroll
            for (int i = 0; i < kSelWaves; ++i) c += counts[side][i];
            side ^= 1;
            if (c >= m) lo = mid;
            else hi = mid - 1;
            exact = c == m;
        }
    }
    __syncthreads();
    // kept: above lo, and the first `ties` of those equal to it; lane i counts
    // both in the wave's i-th group of 64
    if (m == 0) lo = kEnd - 1;
    int up = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        // ballots of the whole wave, so outside any choice of lanes
        const int ups = __popcll(__ballot(key[i] > lo)), eqs = __popcll(__ballot(key[i] == lo && m > 0));
        if (lane == i) {
            up = ups;
            eq = eqs;
        }
    }
    if (lane < NPT) {
        above[lane * kSelWaves + wave] = up;
        equal[lane * kSelWaves + wave] = eq;
    }
    __syncthreads();
    if (wave == 0) {                   // counts before each group, in the order of the tokens
        constexpr int PER = NPT * kSelWaves / 64;
        int before_up[PER], before_eq[PER], sum_up = 0, sum_eq = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            before_up[i] = sum_up;
            before_eq[i] = sum_eq;
            sum_up += above[lane * PER + i];
            sum_eq += equal[lane * PER + i];
        }
        int at_up = sum_up, at_eq = sum_eq;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(at_up, o), y = __shfl_up(at_eq, o);
            at_up += lane >= o ? x : 0;
            at_eq += lane >= o ? y : 0;
        }
        if (lane == 63) counts[0][0] = a.keep - at_up;         // of the equal ones
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            above[lane * PER + i] = at_up - sum_up + before_up[i];
            equal[lane * PER + i] = at_eq - sum_eq + before_eq[i];
        }
    }
    __syncthreads();
    const int ties = counts[0][0];
    if (lane < NPT) {
        up = above[lane * kSelWaves + wave];
        eq = equal[lane * kSelWaves + wave];
    }
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        const bool is_up = key[i] > lo, is_eq = key[i] == lo && m > 0;
        const uint64_t up_mask = __ballot(is_up), eq_mask = __ballot(is_eq);
        const int eq_at = __builtin_amdgcn_readlane(eq, i) +
                          __builtin_amdgcn_mbcnt_hi((uint32_t)(eq_mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)eq_mask, 0));
        const int at = __builtin_amdgcn_readlane(up, i) + min(eq_at, ties) +
                       __builtin_amdgcn_mbcnt_hi((uint32_t)(up_mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)up_mask, 0));
        if (is_up || (is_eq && eq_at < ties)) {
            kept[at] = i * kSelThreads + tid;
            new_w[at] = v[i];
        }
    }
}

// ---- rows beyond 32768 tokens

// Range of the tokens that compete by weight, per (sequence, head) row.
__global__ __launch_bounds__(kThreads) void kv8_evict_ranges_kernel(EvictArgs a, int32_t* begin, int32_t* end) {
    const int row = blockIdx.x * kThreads + threadIdx.x;
    if (row >= a.B * a.c.Hkv) return;
    const int n = evict_len(a, row / a.c.Hkv);
    begin[row] = a.sinks;
    end[row] = n <= a.keep ? a.sinks : n - a.recent;
}

// kept, new_weights and new_lens from the selected middle tokens (ascending).
__global__ __launch_bounds__(kThreads) void kv8_evict_list_kernel(EvictArgs a, const int32_t* __restrict__ indices,
                                                                  int middle) {
    const int groups = (a.keep + kThreads - 1) / kThreads;
    const int row = blockIdx.x / groups, j = blockIdx.x % groups * kThreads + threadIdx.x;
    const int b = row / a.c.Hkv, n = evict_len(a, b);
    if (j == 0 && row == b * a.c.Hkv) a.new_lens[b] = min(n, a.keep);
    if (j >= a.keep) return;
    int s = j;
    if (j >= n) s = -1;
    else if (n > a.keep && j >= a.sinks)
        s = j < a.sinks + middle ? indices[(long)row * middle + j - a.sinks] : n - a.keep + j;
    a.kept[(long)row * a.keep + j] = s;
    a.new_weights[(long)row * a.keep + j] = s < 0 ? 0.0f : a.weights[(long)row * a.width + s];
}

// ---- moving

// One workgroup per (sequence, head, new page), its keys and its values: the
// rows of the kept tokens are looked up once, by one thread each, and then read
// once into registers as codes.
template <int CH>
__global__ __launch_bounds__(kThreads) void kv8_move_kernel(EvictArgs a, int pages) {
    __shared__ float part[2][4];
    __shared__ int src_row[128];
    __shared__ float src_scale[2][128];
    const int j = blockIdx.x % pages;
    const int row = blockIdx.x / pages;
    const int h = row % a.c.Hkv, b = row / a.c.Hkv;
    const int shift = a.c.page_shift, page = 1 << shift, D = a.c.D;
    const int first = j << shift;
    const int here = min(page, min(evict_len(a, b), a.keep) - first);
    if (here <= 0) return;
    const int pid = a.new_table[(long)b * a.new_max_pages + j];
    if (pid < 0 || pid >= a.c.num_pages) return;
    if (threadIdx.x < here) {
        const int s = a.kept[(long)row * a.keep + first + threadIdx.x];
        const int old = s < 0 || s >= evict_len(a, b) ? -1 : a.c.table[(long)b * a.c.max_pages + (s >> shift)];
        const bool there = old >= 0 && old < a.c.num_pages;
        const long at = (long)(there ? old : 0) * a.c.Hkv + h;
        src_row[threadIdx.x] = there ? (int)((at << shift) + (s & (page - 1))) : -1;
        src_scale[0][threadIdx.x] = there ? a.c.k_scale[at] : 0.0f;
        src_scale[1][threadIdx.x] = there ? a.c.v_scale[at] : 0.0f;
    }
    __syncthreads();

    const int per_row = D >> 4;                       // pieces of 16 codes
    const int pieces = here * per_row;
    // the largest code of a row is found first, its scale multiplied once
    u32x4 raw[2][CH];
    float scales[2][CH], top[2] = {0.0f, 0.0f};
    bool infinite = false;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * kThreads + threadIdx.x;
        const int r = min(i, pieces - 1) / per_row, p = i - r * per_row;
        const int at = src_row[r];
        const bool in = i < pieces && at >= 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            raw[x][c] = u32x4{0, 0, 0, 0};
            scales[x][c] = src_scale[x][r];
            if (in) raw[x][c] = *reinterpret_cast<const u32x4*>((x ? a.c.v : a.c.k) + (long)at * D + p * 16);
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float most = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float f[4];
                e4m3_quad_to_f32(raw[x][c][w], f);
                most = fmaxf(fmaxf(most, fmaxf(fabsf(f[0]), fabsf(f[1]))), fmaxf(fabsf(f[2]), fabsf(f[3])));   // no NaN
            }
            top[x] = finite_top(top[x], most * scales[x][c]);
            infinite |= !(fabsf(scales[x][c] * kE4M3Max) < kInf);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) top[x] = fmaxf(top[x], __shfl_xor(top[x], o));
        if ((threadIdx.x & 63) == 0) part[x][threadIdx.x >> 6] = top[x];
    }
    __syncthreads();
    const long to = (long)pid * a.c.Hkv + h;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const float scale = page_scale(fmaxf(fmaxf(part[x][0], part[x][1]), fmaxf(part[x][2], part[x][3])));
        if (threadIdx.x == 0) (x ? a.c.v_scale : a.c.k_scale)[to] = scale;
        uint8_t* codes = (x ? a.c.v : a.c.k) + ((to * D) << shift);
        // the new scale is a power of two: dividing by it is exact, before or after
        // the product with the code
        const float inv = 1.0f / scale;
        auto write = [&](auto saturate) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = c * kThreads + threadIdx.x;
                if (i < pieces) {
                    const float by = saturate ? scales[x][c] : scales[x][c] * inv, then = saturate ? inv : 1.0f;
                    u32x4 o;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        float f[4];
                        e4m3_quad_to_f32(raw[x][c][w], f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = f[e] * by * then;
                        o[w] = e4m3_quad<saturate>(f);
                    }
                    *reinterpret_cast<u32x4*>(codes + (long)i * 16) = o;
                }
            }
        };
        if (__any(infinite)) write(std::true_type{});
        else write(std::false_type{});
    }
}

}  // namespace

hipError_t launch_kv8_append(const AppendArgs& p) {
    return p.dtype == LIX_BF16 ? launch_append<__bf16>(p) : launch_append<_Float16>(p);
}

hipError_t launch_kv8_evict(const EvictArgs& p, const EvictLayout& ly) {
    const int rows = p.B * p.c.Hkv;
    const long cap = (long)p.c.max_pages << p.c.page_shift;
    if (!ly.by_topk) {
        auto select = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(rows), dim3(kSelThreads), 0, p.stream, p);
        };
        if (cap <= 4 * kSelThreads) select(kv8_select_kernel<4>);
        else if (cap <= 16 * kSelThreads) select(kv8_select_kernel<16>);
        else select(kv8_select_kernel<32>);
    } else {
        char* ws = static_cast<char*>(p.workspace);
        int32_t* indices = reinterpret_cast<int32_t*>(ws + ly.indices);
        if (ly.middle > 0) {
            int32_t* begin = reinterpret_cast<int32_t*>(ws + ly.begin);
            int32_t* end = reinterpret_cast<int32_t*>(ws + ly.end);
            hipLaunchKernelGGL(kv8_evict_ranges_kernel, dim3((rows + kThreads - 1) / kThreads), dim3(kThreads), 0,
                               p.stream, p, begin, end);
            TopkArgs t{p.weights, 1, rows, p.width, 1, ly.middle, begin, end, reinterpret_cast<float*>(ws + ly.scores),
                       indices, p.stream};
            const hipError_t e = launch_topk_rows(t);
            if (e != hipSuccess) return e;
        }
        const long groups = (long)rows * ((p.keep + kThreads - 1) / kThreads);
        hipLaunchKernelGGL(kv8_evict_list_kernel, dim3((unsigned)groups), dim3(kThreads), 0, p.stream, p, indices,
                           ly.middle);
    }
    const int page = 1 << p.c.page_shift;
    // no sequence keeps more than it can hold
    const int pages = (int)(((p.keep < cap ? p.keep : cap) + page - 1) / page);
    auto move = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((long)rows * pages)), dim3(kThreads), 0, p.stream, p, pages);
    };
    const int pieces = page * p.c.D / 16;
    if (pieces <= kThreads) move(kv8_move_kernel<1>);
    else if (pieces <= 2 * kThreads) move(kv8_move_kernel<2>);
    else move(kv8_move_kernel<8>);
    return hipGetLastError();
}

}  // namespace lix
