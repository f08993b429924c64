// Softmax attention over the 8-bit cache (lix_kv8_attention): few rows, and
// the joining of parts.
//
// A wave owns 16 NT rows (queries x heads of one key head; for given indices
// the heads of one query) and a part of the keys, and passes over its keys
// once, 32 at a time (kv8_rows.h).  Everything stays in registers: keys and
// values are loaded straight in operand order (kv8_core.h), the next 32 while
// the present ones are used, and waves share nothing, so there is no LDS and no
// barrier.
//
// Few rows: the keys are split into parts (attend_plan) whose (m, l, acc) go
// to the workspace and are joined by a second kernel.
#include <hip/hip_runtime.h>

#include "kv8_rows.h"

namespace lix {

namespace {

// ---------------------------------------------------------------- all visible tokens

template <class Q, int D, int NT>
__global__ __launch_bounds__(256, 2) void kv8_dense_kernel(AttendArgs a, AttendPlan plan) {
    const Task k = wave_task<NT, false>(a, plan);
    if (!k.live) return;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int shift = a.c.page_shift;
    const int len = cached_len(a.c, k.b);

    // rows see more keys the later their query; a padded one sees none
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

    const int chunk = ((most + plan.parts - 1) / plan.parts + 31) & ~31;
    const int lo = min((long)k.part * chunk, (long)most), hi = min((long)lo + chunk, (long)most);

    Rows<Q, D, NT> w;
    w.init();
    if (lo < hi) {
        load_queries<Q, D, NT, false>(a, k, w);
        const int32_t* table = a.c.table + (long)k.b * a.c.max_pages;
        const uint32_t k_off = (lane & 15) * D + 16 * g, v_off = 4 * g * D + (lane & 15) * (D / 16);
        Raw<D> next;
        Scales<2, false> nsc;
        bool nok[2];
        auto load = [&](int s0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int s = s0 + 16 * h;
                const int nth = s >> shift;
                int pid = nth < a.c.max_pages ? table[nth] : -1;
                nok[h] = s < hi && pid >= 0 && pid < a.c.num_pages;
                pid = __builtin_amdgcn_readfirstlane(nok[h] ? pid : 0);
                const long at = (long)pid * a.c.Hkv + k.kvh;
                const long first = ((at << shift) + (s & ((1 << shift) - 1))) * D;
                const uint8_t* kp = a.c.k + first;
                const uint8_t* vp = a.c.v + first;
#pragma unroll
                for (int u = 0; u < D / 64; ++u)
                    next.k[h][u] = *reinterpret_cast<const u32x4*>(kp + k_off + 64u * u);
#pragma unroll
                for (int j = 0; j < 4; ++j) load_values<D>(vp + v_off + (uint32_t)(j * D), next, 4 * h + j);
                nsc.c[h] = nok[h] ? a.c.k_scale[at] : 0.0f;
                nsc.r[h] = nok[h] ? a.c.v_scale[at] : 0.0f;
            }
        };
        load(lo);
        for (int s0 = lo; s0 < hi; s0 += 32) {
            Raw<D> raw = next;
            Scales<2, false> sc = nsc;
            const bool whole = nok[0] && nok[1];
            uint32_t ok = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (nok[j / 4] && s0 + 16 * (j / 4) + 4 * g + j % 4 < hi) ok |= 1u << j;
            if (s0 + 32 < hi) load(s0 + 32);
            w.raise_ref(fmaxf(sc.r[0], sc.r[1]));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sc.c[h] *= a.q.scale_log2;
                dense_ratio(sc.r[h], w.ref, sc.r[h], sc.inv[h]);
            }
            int left[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) left[n] = vis[n] - s0;
            const bool edge = !(whole && s0 + 32 <= least && s0 + 32 <= hi);
            const bool nans = edge && clear_hidden(raw, ok);
            step<Q, D, NT, 2, false>(w, OwnKeys<Q, D>{raw}, sc, edge, left, ok, nans);
        }
    }
    store_rows<Q, D, NT, false>(a, plan, k, w);
}

// ---------------------------------------------------------------- given tokens

template <class Q, int D, int NT>
__global__ __launch_bounds__(256, 2) void kv8_selected_kernel(AttendArgs a, AttendPlan plan) {
    const Task k = wave_task<NT, true>(a, plan);
    if (!k.live) return;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int shift = a.c.page_shift;
    const int seen = visible_tokens(a.q, k.b, k.t, cached_len(a.c, k.b));
    const int chunk = ((a.topk + plan.parts - 1) / plan.parts + 31) & ~31;
    const int lo = (int)min((long)k.part * chunk, (long)a.topk), hi = min(lo + chunk, a.topk);

    Rows<Q, D, NT> w;
    w.init();
    if (lo < hi && seen > 0) {
        load_queries<Q, D, NT, true>(a, k, w);
        const int32_t* table = a.c.table + (long)k.b * a.c.max_pages;
        const int32_t* list = a.indices + ((long)k.b * a.q.S + k.t) * a.topk;
        Raw<D> next;
        Scales<2, true> nsc;
        uint32_t nok = 0;
        bool nall = false;
        auto load = [&](int s0) {
            // entry s0 + lane % 32 of this lane, then passed to where it is used
            const int e = s0 + (lane & 31);
            int idx = e < hi ? list[e] : -1;
            if (idx >= seen) idx = -1;
            int pid = idx >= 0 ? table[idx >> shift] : -1;
            const bool good = pid >= 0 && pid < a.c.num_pages;
            pid = good ? pid : 0;
            const long at = (long)pid * a.c.Hkv + k.kvh;
            const int row = good ? (int)((at << shift) + (idx & ((1 << shift) - 1))) : 0;
            const float ks = good ? a.c.k_scale[at] : 0.0f, vs = good ? a.c.v_scale[at] : 0.0f;
            const uint32_t goods = (uint32_t)__ballot(good);
            nall = goods == 0xffffffffu;
            nok = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const long kr = __shfl(row, 16 * h + (lane & 15));
                const uint8_t* kp = a.c.k + kr * D + 16 * g;
#pragma unroll
                for (int u = 0; u < D / 64; ++u) next.k[h][u] = *reinterpret_cast<const u32x4*>(kp + 64 * u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int from = 16 * h + 4 * g + j;
                    const long vr = __shfl(row, from);
                    load_values<D>(a.c.v + vr * D + (lane & 15) * (D / 16), next, 4 * h + j);
                    nsc.c[4 * h + j] = __shfl(ks, from);
                    nsc.r[4 * h + j] = __shfl(vs, from);
                    nok |= (goods >> from & 1u) << (4 * h + j);
                }
            }
        };
        load(lo);
        for (int s0 = lo; s0 < hi; s0 += 32) {
            Raw<D> raw = next;
            Scales<2, true> sc = nsc;
            const uint32_t ok = nok;
            const bool whole = nall;
            if (s0 + 32 < hi) load(s0 + 32);
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, sc.r[j]);
            if (__any(top > w.ref)) w.raise_ref(column_max(top));
            const float inv = w.ref > 0.0f ? 1.0f / w.ref : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sc.c[j] *= a.q.scale_log2;
                sc.r[j] *= inv;
            }
            const int none[NT] = {};
            if (!whole) clear_hidden(raw, ok);        // all rows see the same keys: no NaN to keep from any
            step<Q, D, NT, 2, true>(w, OwnKeys<Q, D>{raw}, sc, !whole, none, ok, false);
        }
    }
    store_rows<Q, D, NT, true>(a, plan, k, w);
}

// ---------------------------------------------------------------- joining the parts

// One wave per row: weights 2^(m - max m) of its parts, then D / 64 dimensions
// a lane.
template <class Q, int D>
__global__ __launch_bounds__(256) void kv8_join_kernel(AttendArgs a, AttendPlan plan, bool sel) {
    const int lane = threadIdx.x & 63;
    const long r = (long)blockIdx.x * 4 + (threadIdx.x >> 6);      // [b, t, head]
    if (r >= (long)a.q.B * a.q.S * a.q.Hq) return;
    const int head = (int)(r % a.q.Hq);
    const long bt = r / a.q.Hq;
    const int t = (int)(bt % a.q.S), b = (int)(bt / a.q.S);
    Task k;
    k.b = b;
    k.kvh = head / a.q.G;
    k.t = t;
    k.rows = sel ? a.q.G : a.q.S * a.q.G;
    k.part = 0;
    const int row = sel ? head % a.q.G : t * a.q.G + head % a.q.G;
    const long slot0 = part_slot(a, plan, k, row, sel);
    const long all = plan.tasks * plan.parts * k.rows;
    const float* ms = a.workspace + all * D;
    const float* ls = ms + all;

    float top = kNoMax;
    for (int p = lane; p < plan.parts; p += 64) top = fmaxf(top, ms[slot0 + (long)p * k.rows]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    float l = 0.0f;
    float acc[D / 64] = {};
    for (int p = 0; p < plan.parts; ++p) {
        const long slot = slot0 + (long)p * k.rows;
        const float lp = ls[slot];
        if (lp == 0.0f) continue;
        const float f = __builtin_amdgcn_exp2f(ms[slot] - top);
        l += lp * f;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) acc[u] += a.workspace[slot * D + 64 * u + lane] * f;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    typename Q::elem* dst = static_cast<typename Q::elem*>(a.out) + r * D;
#pragma unroll
    for (int u = 0; u < D / 64; ++u) dst[64 * u + lane] = (typename Q::elem)(acc[u] * inv);
    if (lane == 0) a.lse[r] = (top - kLift + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
}

template <class Q, int D>
hipError_t launch(const AttendArgs& a, const AttendPlan& plan) {
    const bool sel = a.indices != nullptr;
    const long units = (long)(sel ? a.q.S : 1) * plan.row_tiles * plan.parts;
    const long grid = (long)a.q.B * a.c.Hkv * ((units + 3) / 4);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, a.stream, a, plan);
    };
    if (plan.waves > 0) {
        const hipError_t e = launch_kv8_tiles(a, plan);
        if (e != hipSuccess) return e;
    } else if (plan.tiles == 2) {
        if constexpr (D <= 128) go(kv8_dense_kernel<Q, D, 2>);
    } else sel ? go(kv8_selected_kernel<Q, D, 1>) : go(kv8_dense_kernel<Q, D, 1>);
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
