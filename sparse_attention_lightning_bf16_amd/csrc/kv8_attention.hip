// Softmax attention over the 8-bit cache (lix_kv8_attention).
//
// A wave owns 16 NT rows (queries x heads of one key head; for given indices
// the heads of one query) and a part of the keys, and passes over its keys
// once, 32 at a time, with a running maximum m and sum l per row:
//     y = scale log2(e) k_scale (q . code)          p = 2^(y - m + 8)
//     l += p        acc += fp16(p v_scale / ref) code        out = acc ref / l
// Everything stays in registers: keys and values are loaded straight in
// operand order (kv8_core.h), the next 32 while the present ones are used, and
// waves share nothing, so there is no LDS and no barrier.
//
// p is at most 2^14 (m moves only when a score passes it by 6, so that the
// accumulators are rarely rescaled) and rounded once to fp16: 11 bits of each
// weight, and weights down to 2^-32 of the largest.  ref is a running bound of
// the v_scale seen, kept 8 times above the largest, so that p v_scale / ref
// stays in fp16's range whatever the scales are.
//
// Hidden keys of a step that has any are masked after the product (y = -inf) and
// the codes of keys that no row sees are cleared, so that stale bytes, NaN
// among them, reach no sum.  A NaN code that some rows see and others do not
// is taken out of the product and added to the rows that see it.
//
// Few rows: the keys are split into parts (attend_plan) whose (m, l, acc) go
// to the workspace and are joined by a second kernel.
#include <hip/hip_runtime.h>

#include "kv8_core.h"

namespace lix {

namespace {

constexpr float kLift = 8.0f;          // weights are held as 2^8 p
constexpr float kSlack = 6.0f;         // a score may pass m by this before m moves
constexpr float kRefRoom = 8.0f;       // ref above the largest v_scale

// 32 keys of a wave: the key codes of two 16-key tiles and the value codes of
// the lane's eight keys.
template <int D>
struct Raw {
    u32x4 k[2][D / 64];
    uint32_t v[D / 64][8];             // [4-byte group of the lane's D / 16 codes][key]
};

template <int D>
__device__ __forceinline__ void load_values(const uint8_t* __restrict__ p, Raw<D>& r, int j) {
    if constexpr (D == 64) {
        r.v[0][j] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (D == 128) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        r.v[0][j] = w.x;
        r.v[1][j] = w.y;
    } else {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int u = 0; u < 4; ++u) r.v[u][j] = w[u];
    }
}

// Rows of a wave and what they have accumulated.
template <class Q, int D, int NT>
struct Rows {
    static constexpr int KS = D / 32;              // steps of the score product
    static constexpr int ET = D / 16;              // output tiles of 16 dimensions
    typename Q::frag q[NT][KS];
    f32x4 acc[ET][NT];
    float m[NT], l[NT];
    float ref;

    __device__ __forceinline__ void init() {
        const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = neg_inf();
            l[n] = 0.0f;
#pragma unroll
            for (int e = 0; e < ET; ++e) acc[e][n] = z;
        }
        ref = 0.0f;
    }
    // Values of largest scale `top` are coming: accumulators go to its unit.
    __device__ __forceinline__ void raise_ref(float top) {
        if (!(top > ref)) return;
        const float next = top * kRefRoom, f = ref / next;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < ET; ++e) acc[e][n] *= f;
        ref = next;
    }
    __device__ __forceinline__ void raise_max(int n, float top) {
        const float next = fmaxf(m[n], column_max(top));
        const float f = next == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(m[n] - next);
        m[n] = next;
        l[n] *= f;
#pragma unroll
        for (int e = 0; e < ET; ++e) acc[e][n] *= f;
    }
};

// Scales of a step: one per 16-key tile (dense) or one per key (indices).
template <bool SEL>
struct Scales {
    float c[SEL ? 8 : 2];              // scale log2(e) k_scale
    float r[SEL ? 8 : 2];              // v_scale, then v_scale / ref
};

// One step of 32 keys.  edge (uniform): some key is hidden from some row; ok
// is then a mask of this lane's eight keys that exist at all, and vis[n] the
// number of keys that the row sees, counted from the step's first (dense).
template <class Q, int D, int NT, bool SEL>
__device__ __forceinline__ void step(Rows<Q, D, NT>& w, Raw<D>& raw, const Scales<SEL>& sc, bool edge,
                                     const int (&vis)[NT], uint32_t ok) {
    constexpr int KS = D / 32;
    const int g = (threadIdx.x & 63) >> 4;
    f32x4 s[2][NT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n) s[h][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const u32x4 kw = raw.k[h][ks / 2];
            const auto a = key_frag<Q>(kw[2 * (ks & 1)], kw[2 * (ks & 1) + 1]);
#pragma unroll
            for (int n = 0; n < NT; ++n) s[h][n] = Q::mfma(a, w.q[n][ks], s[h][n]);
        }

    f16x8 p[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = s[j / 4][n][j % 4] * sc.c[SEL ? j : j / 4];
        if (edge) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool see = (ok >> j & 1) && (SEL || 16 * (j / 4) + 4 * g + j % 4 < vis[n]);
                y[j] = see ? y[j] : neg_inf();       // p = 0 below
            }
        }
        float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
        if (__any(top > w.m[n] + kSlack)) w.raise_max(n, top);
        const float base = (w.m[n] == neg_inf() ? 0.0f : -w.m[n]) + kLift;
        f32x2v pv[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float x = __builtin_amdgcn_exp2f(y[j] + base);
            w.l[n] += x;
            x *= sc.r[SEL ? j : j / 4];
            pv[j / 2][j & 1] = x;
        }
        u32x4 bits;
#pragma unroll
        for (int j = 0; j < 4; ++j) bits[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pv[j], f16x2));
        p[n] = __builtin_bit_cast(f16x8, bits);
    }

    if (edge) {
        uint32_t any_nan = 0;
#pragma unroll
        for (int u = 0; u < D / 64; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                raw.v[u][j] = ok >> j & 1 ? raw.v[u][j] : 0u;
                any_nan |= nan_codes(raw.v[u][j]);
            }
        if (!SEL && __any(any_nan != 0)) {
            // rare: 1 where a code is NaN times 1 where a row sees the key
            f16x8 seen[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    seen[n][j] = 16 * (j / 4) + 4 * g + j % 4 < vis[n] ? (_Float16)1.0f : (_Float16)0.0f;
#pragma unroll
            for (int u = 0; u < D / 64; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    __builtin_amdgcn_sched_barrier(0);
                    f16x8 bad;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t byte = raw.v[u][j] >> (8 * e) & 0x7fu;
                        bad[j] = byte == 0x7fu ? (_Float16)1.0f : (_Float16)0.0f;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const f32x4 hit = QFp16::mfma(bad, seen[n], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (hit[i] > 0.0f) w.acc[4 * u + e][n][i] = __uint_as_float(0x7fc00000u);
                    }
                }
#pragma unroll
            for (int u = 0; u < D / 64; ++u)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t bad = nan_codes(raw.v[u][j]) >> 7;      // 1 in each NaN byte
                    raw.v[u][j] &= ~(bad * 0xffu);
                }
        }
    }
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
        f16x8 f[4];
        value_frags(raw.v[u], f);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int n = 0; n < NT; ++n) w.acc[4 * u + e][n] = QFp16::mfma(f[e], p[n], w.acc[4 * u + e][n]);
    }
}

// What a wave works on.
struct Task {
    int b, kvh;
    int t;                             // the query, with indices
    int row0, rows;                    // first row of the wave, rows of the group
    int part;
    bool live;
};

template <int NT, bool SEL>
__device__ __forceinline__ Task wave_task(const AttendArgs& a, const AttendPlan& plan) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Task k;
    const long pairs = (long)a.q.B * a.c.Hkv;
    const long block = blockIdx.x;
    const long pair = block % pairs;
    long u = block / pairs * 4 + wave;             // (row tile, part) of the pair, part fastest
    const int groups = SEL ? a.q.S : 1;
    const long units = (long)groups * plan.row_tiles * plan.parts;
    k.live = u < units;
    k.b = (int)(pair / a.c.Hkv);
    k.kvh = (int)(pair % a.c.Hkv);
    k.part = (int)(u % plan.parts);
    u /= plan.parts;
    if (SEL) {
        k.row0 = (int)(u % plan.row_tiles) * 16 * NT;
        k.t = (int)(u / plan.row_tiles);
        k.rows = a.q.G;
    } else {
        // late rows see the most keys: they go first
        k.row0 = (plan.row_tiles - 1 - (int)u) * 16 * NT;
        k.t = 0;
        k.rows = a.q.S * a.q.G;
    }
    return k;
}

// Query and head of row r of the wave's group.
template <bool SEL>
__device__ __forceinline__ void row_of(const AttendArgs& a, const Task& k, int r, int& t, int& head) {
    t = SEL ? k.t : r / a.q.G;
    head = k.kvh * a.q.G + (SEL ? r : r - t * a.q.G);
}

template <class Q, int D, int NT, bool SEL>
__device__ __forceinline__ void load_queries(const AttendArgs& a, const Task& k, Rows<Q, D, NT>& w) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const typename Q::elem* q = static_cast<const typename Q::elem*>(a.q.q);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = k.row0 + 16 * n + (lane & 15);
        int t, head;
        row_of<SEL>(a, k, min(r, k.rows - 1), t, head);
        const typename Q::elem* at = q + k.b * a.q.sb + t * a.q.ss + head * a.q.sh + 16 * g;
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks)
            w.q[n][ks] = *reinterpret_cast<const typename Q::frag*>(at + 64 * (ks / 2) + 8 * (ks & 1));
    }
}

// Workspace of part results: acc [tasks][parts][D] fp32 of every row of the
// group, then m and l.  slot = ((pair, query group), part, row).
__device__ __forceinline__ long part_slot(const AttendArgs& a, const AttendPlan& plan, const Task& k, int r, bool sel) {
    const long group = sel ? ((long)(k.b * a.c.Hkv + k.kvh) * a.q.S + k.t) : (long)(k.b * a.c.Hkv + k.kvh);
    return (group * plan.parts + k.part) * k.rows + r;
}

// Rows of the wave: written out, or its part to the workspace.
template <class Q, int D, int NT, bool SEL>
__device__ __forceinline__ void store_rows(const AttendArgs& a, const AttendPlan& plan, const Task& k,
                                           Rows<Q, D, NT>& w) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    typedef typename Q::elem E;
    typedef E e4 __attribute__((ext_vector_type(4)));
    const long all = plan.tasks * plan.parts * k.rows;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float l = column_sum(w.l[n]);
        const int r = k.row0 + 16 * n + (lane & 15);
        if (r >= k.rows) continue;
        // c[i] of tile e is dimension (4 g + i) D / 16 + e: D / 4 consecutive ones
        if (plan.parts > 1) {
            const long slot = part_slot(a, plan, k, r, SEL);
            float* dst = a.workspace + slot * D + g * (D / 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < D / 16; e += 4) {
                    f32x4 o;
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[x] = w.acc[e + x][n][i] * w.ref;
                    *reinterpret_cast<f32x4*>(dst + i * (D / 16) + e) = o;
                }
            if (g == 0) {
                a.workspace[all * D + slot] = w.m[n];
                a.workspace[all * (D + 1) + slot] = l;
            }
        } else {
            int t, head;
            row_of<SEL>(a, k, r, t, head);
            const long row = ((long)k.b * a.q.S + t) * a.q.Hq + head;
            const float f = l == 0.0f ? 0.0f : w.ref / l;
            E* dst = static_cast<E*>(a.out) + row * D + g * (D / 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < D / 16; e += 4) {
                    e4 o;
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[x] = (E)(w.acc[e + x][n][i] * f);
                    *reinterpret_cast<e4*>(dst + i * (D / 16) + e) = o;
                }
            if (g == 0) a.lse[row] = (w.m[n] - kLift + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
        }
    }
}

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
        Scales<false> nsc;
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
            Scales<false> sc = nsc;
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
                sc.r[h] = w.ref > 0.0f ? sc.r[h] / w.ref : 0.0f;
            }
            int left[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) left[n] = vis[n] - s0;
            step<Q, D, NT, false>(w, raw, sc, !(whole && s0 + 32 <= least && s0 + 32 <= hi), left, ok);
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
        Scales<true> nsc;
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
            Scales<true> sc = nsc;
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
            step<Q, D, NT, true>(w, raw, sc, !whole, none, ok);
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

    float top = neg_inf();
    for (int p = lane; p < plan.parts; p += 64) top = fmaxf(top, ms[slot0 + (long)p * k.rows]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float ref = top == neg_inf() ? 0.0f : top;
    float l = 0.0f;
    float acc[D / 64] = {};
    for (int p = 0; p < plan.parts; ++p) {
        const long slot = slot0 + (long)p * k.rows;
        const float lp = ls[slot];
        if (lp == 0.0f) continue;
        const float f = __builtin_amdgcn_exp2f(ms[slot] - ref);
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
    if constexpr (D <= 128) {
        if (plan.tiles == 2) sel ? go(kv8_selected_kernel<Q, D, 2>) : go(kv8_dense_kernel<Q, D, 2>);
    }
    if (plan.tiles == 1) sel ? go(kv8_selected_kernel<Q, D, 1>) : go(kv8_dense_kernel<Q, D, 1>);
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
