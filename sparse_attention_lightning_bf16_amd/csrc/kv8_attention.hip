// Softmax attention over the 8-bit cache (lix_kv8_attention): few rows, and
// the joining of parts.
//
// A workgroup owns 16 NT rows (queries x heads of one key head; for given
// indices the heads of one query) and a part of the keys; its four waves take
// turns of 32 keys (kv8_rows.h) and are joined in LDS at the end.  Keys and
// values are loaded straight in operand order (kv8_core.h) into registers, two
// turns ahead, and nothing is shared on the way: no barrier in the loop.
//
// Bound by reading the codes.  The parts (attend_plan) make about twice
// as many workgroups as are resident, so that sequences of different lengths
// even out; their (m, l, acc) go to the workspace and are joined by a second
// kernel.
#include <hip/hip_runtime.h>

#include "kv8_rows.h"

namespace lix {

namespace {

constexpr int kWaves = 4;
constexpr int kTurn = 32 * kWaves;     // keys of a workgroup's turn

// Two turns of codes in registers, where two waves per SIMD have room for them;
// else one.
template <int D, int NT>
constexpr bool kTwoAhead = D * NT <= 128;

// The four waves' rows joined into the first one's.
template <class Q, int D, int NT>
__device__ __forceinline__ void join_waves(Rows<Q, D, NT>& w, int wave, f32x4 (&acc)[2][Rows<Q, D, NT>::ET][NT][64],
                                           float (&ml)[2][2][NT][64]) {
    constexpr int ET = Rows<Q, D, NT>::ET;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < ET; ++e) w.acc[e][n] *= w.ref;
    w.ref = 1.0f;
#pragma unroll
    for (int half = kWaves / 2; half > 0; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < ET; ++e) acc[wave - half][e][n][lane] = w.acc[e][n];
                ml[wave - half][0][n][lane] = w.m[n];
                ml[wave - half][1][n][lane] = w.l[n];
            }
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float m = ml[wave][0][n][lane], next = fmaxf(m, w.m[n]);
                const float mine = __builtin_amdgcn_exp2f(w.m[n] - next), other = __builtin_amdgcn_exp2f(m - next);
                w.m[n] = next;
                w.l[n] = w.l[n] * mine + ml[wave][1][n][lane] * other;
#pragma unroll
                for (int e = 0; e < ET; ++e) w.acc[e][n] = w.acc[e][n] * mine + acc[wave][e][n][lane] * other;
            }
        }
        __syncthreads();
    }
}

// Task of a workgroup: a pair's row tile and part, part fastest.
template <int NT, bool SEL>
__device__ __forceinline__ Task part_task(const AttendArgs& a, const AttendPlan& plan) {
    Task k;
    const long pairs = (long)a.q.B * a.c.Hkv;
    const long block = blockIdx.x;
    const long pair = block % pairs;
    long u = block / pairs;
    k.live = true;
    k.b = (int)(pair / a.c.Hkv);
    k.kvh = (int)(pair % a.c.Hkv);
    k.part = (int)(u % plan.parts);
    u /= plan.parts;
    k.row0 = (int)(u % plan.row_tiles) * 16 * NT;
    k.t = SEL ? (int)(u / plan.row_tiles) : 0;
    k.rows = SEL ? a.q.G : a.q.S * a.q.G;
    return k;
}

// Keys of a part of n: whole turns, at least four of them.
__device__ __forceinline__ void part_range(int n, const AttendPlan& plan, int part, int& lo, int& hi) {
    const int even = (n + plan.parts - 1) / plan.parts;
    const long chunk = max((even + kTurn - 1) / kTurn, 4) * (long)kTurn;
    lo = (int)min(part * chunk, (long)n);
    hi = (int)min(lo + chunk, (long)n);
}

// ---------------------------------------------------------------- all visible tokens

template <class Q, int D, int NT>
__global__ __launch_bounds__(256, 2) void kv8_dense_kernel(AttendArgs a, AttendPlan plan) {
    using R = Rows<Q, D, NT>;
    __shared__ f32x4 sh_acc[2][R::ET][NT][64];
    __shared__ float sh_ml[2][2][NT][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Task k = part_task<NT, false>(a, plan);
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int shift = a.c.page_shift;
    const int len = cached_len(a.c, k.b);

    // keys [0, most) are seen by some row, [0, least) by all
    const int last = min(k.row0 + 16 * NT, k.rows) - 1;
    int most = 0, least = len;
    int vis[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = min(k.row0 + 16 * n + (lane & 15), last);
        vis[n] = visible_tokens(a.q, k.b, r / a.q.G, len);
        most = max(most, vis[n]);
        least = min(least, vis[n]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        most = max(most, __shfl_xor(most, o));
        least = min(least, __shfl_xor(least, o));
    }
    most = __builtin_amdgcn_readfirstlane(most);
    least = __builtin_amdgcn_readfirstlane(least);
    int lo, hi;
    part_range(most, plan, k.part, lo, hi);

    R w;
    w.init();
    const int first = lo + 32 * wave;
    if (first < hi) {
        const int32_t* table = a.c.table + (long)k.b * a.c.max_pages;
        // Lane e looks up entry e of the wave's next 32 turns (two entries of 16
        // tokens each): row and scales, the pages one such batch ahead.
        int token = first + (lane >> 1) * kTurn + 16 * (lane & 1), pid;
        auto find = [&]() { pid = token < hi ? table[token >> shift] : -1; };
        int row = 0;
        uint64_t good = 0;
        float kscale = 0.0f, vscale = 0.0f;
        auto look = [&]() {
            const bool there = pid >= 0 && pid < a.c.num_pages;
            const long at = (long)(there ? pid : 0) * a.c.Hkv + k.kvh;
            row = there ? (int)((at << shift) + (token & ((1 << shift) - 1))) : 0;
            kscale = there ? a.c.k_scale[at] : 0.0f;
            vscale = there ? a.c.v_scale[at] : 0.0f;
            good = __ballot(there);
            token = token < hi ? token + 32 * kTurn : token;
            find();
        };
        float c = 0.0f, r = 0.0f, inv = 0.0f, ref = 0.0f;
        uint64_t used = 0;
        auto use = [&]() {
            float top = vscale;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
            top = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(top)));
            if (top > ref) ref = top * kRefRoom;
            c = kscale * a.q.scale_log2;
            dense_ratio(vscale, ref, r, inv);
            used = good;
            if (ref > w.ref) w.set_ref(ref);
        };

        const uint32_t k_off = (lane & 15) * D + 16 * g, v_off = 4 * g * D + (lane & 15) * (D / 16);
        auto load = [&](Raw<D>& raw, int i) {      // the wave's i-th turn
            const int e = 2 * (i & 31);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const long at = (long)__builtin_amdgcn_readlane(row, e + h) * D;
                const uint8_t *kp = a.c.k + at, *vp = a.c.v + at;
#pragma unroll
                for (int u = 0; u < D / 64; ++u) raw.k[h][u] = *reinterpret_cast<const u32x4*>(kp + (k_off + 64u * u));
#pragma unroll
                for (int j = 0; j < 4; ++j) load_values<D>(vp + (v_off + (uint32_t)(j * D)), raw, 4 * h + j);
            }
        };
        auto compute = [&](Raw<D>& raw, int i) {
            const int s0 = first + i * kTurn, e = 2 * (i & 31);
            const uint32_t there = (uint32_t)(used >> e) & 3;
            const bool edge = there != 3 || s0 + 32 > least || s0 + 32 > hi;
            Scales<2, false> sc;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                auto lane_of = [&](float v) {
                    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), e + h));
                };
                sc.c[h] = lane_of(c);
                sc.r[h] = lane_of(r);
                sc.inv[h] = lane_of(inv);
            }
            uint32_t ok = ~0u;
            int left[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) left[n] = vis[n] - s0;
            if (edge) {
                ok = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) ok |= (there >> (j / 4) & 1) && s0 + key_of(j, g) < hi ? 1u << j : 0u;
                if (clear_hidden(raw, ok)) {
                    mark_nans<Q, D, NT, 2>(w, [&](int, int u, uint32_t (&v)[8]) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = raw.v[u][j];
                    }, left, ok);
#pragma unroll
                    for (int u = 0; u < D / 64; ++u)
#pragma unroll
                        for (int j = 0; j < 8; ++j) raw.v[u][j] = without_nans(raw.v[u][j]);
                }
            }
            step<Q, D, NT, 2, false>(w, OwnKeys<Q, D>{raw}, sc, edge, left, ok);
        };

        const int turns = (hi - first + kTurn - 1) / kTurn;
        find();
        look();
        if constexpr (kTwoAhead<D, NT>) {
            Raw<D> one, two;
            load(one, 0);
            if (turns > 1) load(two, 1);
            load_queries<Q, D, NT, false>(a, k, w);
            // A buffer is loaded again as soon as it has been used: the other is
            // then already on its way.
            for (int i = 0; i < turns; i += 2) {
                if ((i & 31) == 0) use();
                compute(one, i);
                if (i + 2 < turns) {
                    if ((i + 2 & 31) == 0) look();
                    load(one, i + 2);
                }
                if (i + 1 < turns) compute(two, i + 1);
                if (i + 3 < turns) load(two, i + 3);
            }
        } else {
            Raw<D> one;
            load(one, 0);
            load_queries<Q, D, NT, false>(a, k, w);
            for (int i = 0; i < turns; ++i) {
                if ((i & 31) == 0) use();
                compute(one, i);
                if (i + 1 < turns) {
                    if ((i + 1 & 31) == 0) look();
                    load(one, i + 1);
                }
            }
        }
    }
    join_waves<Q, D, NT>(w, wave, sh_acc, sh_ml);
    if (wave == 0) store_rows<Q, D, NT, false>(a, plan, k, w);
}

// ---------------------------------------------------------------- given tokens

template <class Q, int D>
__global__ __launch_bounds__(256, 2) void kv8_selected_kernel(AttendArgs a, AttendPlan plan) {
    using R = Rows<Q, D, 1>;
    __shared__ f32x4 sh_acc[2][R::ET][1][64];
    __shared__ float sh_ml[2][2][1][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Task k = part_task<1, true>(a, plan);
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int shift = a.c.page_shift;
    const int seen = __builtin_amdgcn_readfirstlane(visible_tokens(a.q, k.b, k.t, cached_len(a.c, k.b)));
    int lo, hi;
    part_range(seen > 0 ? a.topk : 0, plan, k.part, lo, hi);

    R w;
    w.init();
    const int first = lo + 32 * wave;
    if (first < hi) {
        const int32_t* table = a.c.table + (long)k.b * a.c.max_pages;
        const int32_t* list = a.indices + ((long)k.b * a.q.S + k.t) * a.topk;
        // lane e looks up entry e of the wave's next two turns
        int at_entry = first + (lane >> 5) * kTurn + (lane & 31);
        auto entry = [&](int e) {
            const int idx = e < hi ? list[e] : -1;
            return idx < seen ? idx : -1;
        };
        auto page_of = [&](int idx) { return idx >= 0 ? table[idx >> shift] : -1; };
        int idx = entry(at_entry), pid = page_of(idx), ahead = entry(at_entry + 2 * kTurn);
        int row = 0;
        float kscale = 0.0f, vscale = 0.0f;
        uint64_t good = 0;
        auto look = [&]() {
            const bool there = pid >= 0 && pid < a.c.num_pages;
            const long at = (long)(there ? pid : 0) * a.c.Hkv + k.kvh;
            row = there ? (int)((at << shift) + (idx & ((1 << shift) - 1))) : 0;
            kscale = there ? a.c.k_scale[at] : 0.0f;
            vscale = there ? a.c.v_scale[at] : 0.0f;
            good = __ballot(there);
            idx = ahead;
            pid = page_of(idx);
            at_entry = at_entry < hi ? at_entry + 2 * kTurn : at_entry;
            ahead = entry(at_entry + 2 * kTurn);
        };
        float c = 0.0f, r = 0.0f, ref = 0.0f;
        uint64_t used = 0;
        auto use = [&]() {
            float top = vscale;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
            top = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(top)));
            if (top > ref) ref = top * kRefRoom;
            c = kscale * a.q.scale_log2;
            r = ref > 0.0f ? vscale * __builtin_amdgcn_rcpf(ref) : 0.0f;
            used = good;
            if (ref > w.ref) w.set_ref(ref);
        };
        auto load = [&](Raw<D>& raw, int i) {      // the wave's i-th turn
            const int e0 = 32 * (i & 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* kp = a.c.k + (long)__shfl(row, e0 + 16 * h + (lane & 15)) * D + 16 * g;
#pragma unroll
                for (int u = 0; u < D / 64; ++u) raw.k[h][u] = *reinterpret_cast<const u32x4*>(kp + 64 * u);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    load_values<D>(a.c.v + (long)__shfl(row, e0 + 16 * h + 4 * g + j) * D + (lane & 15) * (D / 16), raw,
                                   4 * h + j);
            }
        };
        auto compute = [&](Raw<D>& raw, int i) {
            const int e0 = 32 * (i & 1);
            const uint32_t there = (uint32_t)(used >> e0);
            Scales<2, true> sc;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sc.c[j] = __shfl(c, e0 + key_of(j, g));
                sc.r[j] = __shfl(r, e0 + key_of(j, g));
            }
            uint32_t ok = ~0u;
            if (there != ~0u) {
                ok = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) ok |= (there >> key_of(j, g) & 1) << j;
                clear_hidden(raw, ok);             // all rows see the same keys: no NaN to keep from any
            }
            const int none[1] = {};
            step<Q, D, 1, 2, true>(w, OwnKeys<Q, D>{raw}, sc, there != ~0u, none, ok);
        };

        const int turns = (hi - first + kTurn - 1) / kTurn;
        look();
        if constexpr (kTwoAhead<D, 1>) {
            Raw<D> one, two;
            load(one, 0);
            if (turns > 1) load(two, 1);
            load_queries<Q, D, 1, true>(a, k, w);
            for (int i = 0; i < turns; i += 2) {
                use();
                if (i + 2 < turns) look();
                compute(one, i);
                if (i + 2 < turns) load(one, i + 2);
                if (i + 1 < turns) compute(two, i + 1);
                if (i + 3 < turns) load(two, i + 3);
            }
        } else {
            Raw<D> one;
            load(one, 0);
            load_queries<Q, D, 1, true>(a, k, w);
            for (int i = 0; i < turns; ++i) {
                if ((i & 1) == 0) use();
                compute(one, i);
                if (i + 1 < turns) {
                    if (i & 1) look();
                    load(one, i + 1);
                }
            }
        }
    }
    join_waves<Q, D, 1>(w, wave, sh_acc, sh_ml);
    if (wave == 0) store_rows<Q, D, 1, true>(a, plan, k, w);
}

// ---------------------------------------------------------------- joining the parts

// One wave per row.  A lane first holds a part's m and l (up to four of them),
// whose factors 2^(m - max m) / l then go round, while a lane adds up D / 64
// consecutive dimensions; no load waits for another.
template <class Q, int D>
__global__ __launch_bounds__(256) void kv8_join_kernel(AttendArgs a, AttendPlan plan, bool sel) {
    constexpr int N = D / 64;
    typedef float vec __attribute__((ext_vector_type(N)));
    typedef typename Q::elem out_vec __attribute__((ext_vector_type(N)));
    const int lane = threadIdx.x & 63;
    const long r = (long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);      // [b, t, head]
    if (r >= (long)a.q.B * a.q.S * a.q.Hq) return;
    const int head = (int)(r % a.q.Hq);
    const long bt = r / a.q.Hq;
    Task k;
    k.t = (int)(bt % a.q.S);
    k.b = (int)(bt / a.q.S);
    k.kvh = head / a.q.G;
    k.rows = sel ? a.q.G : a.q.S * a.q.G;
    k.part = 0;
    const long slot0 = part_slot(a, plan, k, sel ? head % a.q.G : k.t * a.q.G + head % a.q.G, sel);
    const long all = plan.tasks * plan.parts * k.rows;
    const float* ms = a.workspace + all * D;
    const float* ls = ms + all;

    constexpr int PL = kMaxParts / 64;
    float m[PL], l[PL], top = kNoMax;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int p = 64 * i + lane;
        const bool is = p < plan.parts;
        m[i] = is ? ms[slot0 + (long)p * k.rows] : kNoMax;
        l[i] = is ? ls[slot0 + (long)p * k.rows] : 0.0f;
        top = fmaxf(top, m[i]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        m[i] = __builtin_amdgcn_exp2f(m[i] - top);
        sum += l[i] * m[i];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    vec acc = {};
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int here = min(plan.parts - 64 * i, 64);
        const float* src = a.workspace + (slot0 + 64L * i * k.rows) * D + lane * N;
#pragma unroll 8
        for (int p = 0; p < here; ++p) {
            const float f = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(m[i]), p));
            acc += *reinterpret_cast<const vec*>(src + (long)p * k.rows * D) * f;
        }
    }
    out_vec o;
#pragma unroll
    for (int u = 0; u < N; ++u) o[u] = (typename Q::elem)(acc[u] * inv);
    *reinterpret_cast<out_vec*>(static_cast<typename Q::elem*>(a.out) + r * D + lane * N) = o;
    if (lane == 0) a.lse[r] = (top - kLift + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f;
}

template <class Q, int D>
hipError_t launch(const AttendArgs& a, const AttendPlan& plan) {
    const bool sel = a.indices != nullptr;
    const long grid = plan.tasks * plan.row_tiles * plan.parts;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * kWaves), 0, a.stream, a, plan);
    };
    if (plan.waves > 0) {
        const hipError_t e = launch_kv8_tiles(a, plan);
        if (e != hipSuccess) return e;
    } else if (plan.tiles == 2) {
        if constexpr (D <= 128) go(kv8_dense_kernel<Q, D, 2>);
    } else {
        sel ? go(kv8_selected_kernel<Q, D>) : go(kv8_dense_kernel<Q, D, 1>);
    }
    if (plan.parts > 1) {
        const long rows = (long)a.q.B * a.q.S * a.q.Hq;
        hipLaunchKernelGGL((kv8_join_kernel<Q, D>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, a.stream, a, plan,
                           sel);
    }
    return hipGetLastError();
}

template <class Q>
hipError_t launch_dim(const AttendArgs& a, const AttendPlan& plan) {
    switch (a.c.D) {
        case 64: return launch<Q, 64>(a, plan);
        case 128: return launch<Q, 128>(a, plan);
        default: return launch<Q, 256>(a, plan);
    }
}

}  // namespace

hipError_t launch_kv8_attention(const AttendArgs& a, const AttendPlan& plan) {
    return a.q.dtype == LIX_BF16 ? launch_dim<QBf16>(a, plan) : launch_dim<QFp16>(a, plan);
}

}  // namespace lix
