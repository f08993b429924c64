// Rows of an attention wave (lix_kv8_attention): running maximum and sum of
// the softmax, the step over 32 keys, and what a wave works on and writes.
//
//     y = scale log2(e) k_scale (q . code)          p = 2^(y - m + 8)
//     l += p        acc += fp16(p v_scale / ref) code        out = acc ref / l
//
// ref is a running bound of the v_scale seen, kept 8 times above the largest.
// m moves only when weights p v_scale / ref pass 2^14, so that accumulators are
//  rarely rescaled and the weights stay in fp16's range whatever the scales
// are; each is rounded once to fp16 (11 bits).
//
// Hidden keys of a step that has any are masked after the product (y = -inf)
// and the codes of keys that no row sees are cleared, so that stale bytes, NaN
// among them, reach no sum.  A NaN code that some rows see and others do not
// is taken out of the product and added to the rows that see it.
#pragma once

#include "kv8_core.h"

namespace lix {

constexpr float kLift = 8.0f;          // weights are held as 2^8 p
constexpr float kMost = 16384.0f;      // m moves when four weights times v_scale / ref pass 2^14
constexpr float kRefRoom = 8.0f;       // ref above the largest v_scale
constexpr float kNoMax = -3.0e38f;     // m before any key: any score passes it, 2^(m - score) is 0

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
            m[n] = kNoMax;
            l[n] = 0.0f;
#pragma unroll
            for (int e = 0; e < ET; ++e) acc[e][n] = z;
        }
        ref = 0.0f;
    }
    // Values of largest scale `top` are coming: accumulators go to its unit.
    __device__ __forceinline__ void raise_ref(float top) {
        if (top > ref) set_ref(top * kRefRoom);
    }
    __device__ __forceinline__ void set_ref(float next) {
        const float f = ref / next;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < ET; ++e) acc[e][n] *= f;
        ref = next;
    }
    __device__ __forceinline__ void raise_max(int n, float top) {
        const float next = fmaxf(m[n], column_max(top));
        const float f = __builtin_amdgcn_exp2f(m[n] - next);
        m[n] = next;
        l[n] *= f;
#pragma unroll
        for (int e = 0; e < ET; ++e) acc[e][n] *= f;
    }
};

// Scales of KH tiles of 16 keys: one set per tile (dense) or per key (indices).
template <int KH, bool SEL>
struct Scales {
    float c[SEL ? 4 * KH : KH];        // scale log2(e) k_scale
    float r[SEL ? 4 * KH : KH];        // v_scale / ref (dense: its log2)
    float inv[SEL ? 1 : KH];           // ref / v_scale
};

// v_scale / ref as the dense kernels use it: in the exponent of the weights,
// and divided out of their sum.  Below 2^-60 no weight times a code is left in
// fp16's range; the bound keeps a page of scale zero out of 0 * infinity.
__device__ __forceinline__ void dense_ratio(float v_scale, float ref, float& log2_r, float& inv) {
    const float r = fmaxf(v_scale * __builtin_amdgcn_rcpf(ref), 0x1p-60f);
    log2_r = __builtin_amdgcn_logf(r);
    inv = __builtin_amdgcn_rcpf(r);
}

// Fragments of 32 keys from a wave's own registers.
template <class Q, int D>
struct OwnKeys {
    static constexpr bool kShared = false;
    const Raw<D>& raw;
    __device__ __forceinline__ typename Q::frag key(int h, int ks) const {
        const u32x4 w = raw.k[h][ks / 2];
        return key_frag<Q>(w[2 * (ks & 1)], w[2 * (ks & 1) + 1]);
    }
    __device__ __forceinline__ void values(int, int u, f16x8 (&f)[4]) const { value_frags(raw.v[u], f); }
};

// Key of this lane's slot j = 4 h + i, counted from the first: 16 h + 4 g + i.
__device__ __forceinline__ int key_of(int j, int g) { return 16 * (j / 4) + 4 * g + j % 4; }

// Rare: a NaN among the values of keys that not every row sees.  The products
// are taken without it (0 in its place), and the outputs of the rows that see
// its key become NaN here: 1 where a value is NaN times 1 where a row sees the
// key.  words(q, u, v): the eight codes' words of 32-key group q, as Raw::v.
template <class Q, int D, int NT, int KH, class Words>
__device__ __forceinline__ void mark_nans(Rows<Q, D, NT>& w, const Words& words, const int (&vis)[NT], uint32_t ok) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll 1
    for (int q = 0; q < KH / 2; ++q)
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            __builtin_amdgcn_sched_barrier(0);
            uint32_t v[8];
            words(q, u, v);
            f16x8 seen[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    seen[n][j] = (ok >> (8 * q + j) & 1) && 32 * q + key_of(j, g) < vis[n] ? (_Float16)1.0f
                                                                                          : (_Float16)0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f16x8 bad;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t byte = v[j] >> (8 * e) & 0x7fu;
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
        }
}

// One pass over KH tiles of 16 keys.  edge (uniform): some key is hidden from
// some row; ok is then a mask of this lane's 4 KH keys that exist at all, and
// vis[n] the number of keys that the row sees, counted from the first (dense).
// Codes of keys that no row sees are zero already, and so are NaN codes of
// keys that some rows do not see (mark_nans).
//
// All scores first, then one test whether any of them passes its row's
// maximum, then all weights: the products of a row tile are in flight while
// the weights of another are taken.
template <class Q, int D, int NT, int KH, bool SEL, class Src>
__device__ __forceinline__ void step(Rows<Q, D, NT>& w, const Src& src, const Scales<KH, SEL>& sc, bool edge,
                                     const int (&vis)[NT], uint32_t ok) {
    constexpr int KS = D / 32;
    const int g = (threadIdx.x & 63) >> 4;
    f32x4 s[KH][NT];
#pragma unroll
    for (int h = 0; h < KH; ++h) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[h][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const auto a = src.key(h, ks);
#pragma unroll
            for (int n = 0; n < NT; ++n) s[h][n] = Q::mfma(a, w.q[n][ks], s[h][n]);
        }
    }

    // Operands out of LDS: both products are scheduled as loads and matrix
    // instructions in turns, which keeps the next operands ahead (4096 rows of two
    // sequences up to 8192 long, 32 heads: 860 us without, 785 with; 797 with wave
    // priorities instead).
    if constexpr (Src::kShared) __builtin_amdgcn_iglp_opt(1);
    constexpr int CS = SEL ? 4 * KH : KH;
    float c[CS];                       // what is left to multiply the scores with
#pragma unroll
    for (int j = 0; j < CS; ++j) c[j] = sc.c[j];
    if (edge) {
        // the masks stay inside the branch: hoisted, they cost every step
        int here = g;
        asm volatile("" : "+v"(here), "+v"(ok));
#pragma unroll
        for (int h = 0; h < KH; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool see = (ok >> (4 * h + i) & 1) && (SEL || key_of(4 * h + i, here) < vis[n]);
                    s[h][n][i] = see ? s[h][n][i] * c[SEL ? 4 * h + i : h] : neg_inf();       // p = 0 below
                }
#pragma unroll
        for (int j = 0; j < CS; ++j) c[j] = 1.0f;
    }

    // The weights, and their sums over four keys: no weight is above its sum, so
    // the sums tell whether m has to move.
    f32x4 x[KH][NT];
    float sum[KH][NT];
    auto weights = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < KH; ++h) {
                const float add = (kLift - w.m[n]) + (SEL ? 0.0f : sc.r[h]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[h][n][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[h][n][i], c[SEL ? 4 * h + i : h], add));
                sum[h][n] = (x[h][n][0] + x[h][n][1]) + (x[h][n][2] + x[h][n][3]);
            }
    };
    weights();
    float most = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < KH; ++h) most = fmaxf(most, sum[h][n]);
    if (__any(most > kMost)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float top = kNoMax;
#pragma unroll
            for (int h = 0; h < KH; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, s[h][n][i] * c[SEL ? 4 * h + i : h]);
            w.raise_max(n, top);
        }
        weights();
    }

    f16x8 p[KH / 2][NT], rest[KH / 2][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < KH; ++h) {
            f32x4 v = x[h][n];
            if constexpr (SEL) {
                w.l[n] += sum[h][n];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] *= sc.r[4 * h + i];
            } else {
                w.l[n] = __builtin_fmaf(sum[h][n], sc.inv[h], w.l[n]);
            }
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                f32x2v two = {v[i], v[i + 1]};
                const f16x2 hi = __builtin_convertvector(two, f16x2);
                p[h / 2][n][4 * (h & 1) + i] = hi[0];
                p[h / 2][n][4 * (h & 1) + i + 1] = hi[1];
                if constexpr (Q::kTwoWeights) {
                    two[0] -= (float)hi[0];
                    two[1] -= (float)hi[1];
                    const f16x2 lo = __builtin_convertvector(two, f16x2);
                    rest[h / 2][n][4 * (h & 1) + i] = lo[0];
                    rest[h / 2][n][4 * (h & 1) + i + 1] = lo[1];
                }
            }
        }

    if constexpr (Src::kShared) __builtin_amdgcn_iglp_opt(1);
#pragma unroll
    for (int q = 0; q < KH / 2; ++q)
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            f16x8 f[4];
            src.values(q, u, f);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    w.acc[4 * u + e][n] = QFp16::mfma(f[e], p[q][n], w.acc[4 * u + e][n]);
                    if constexpr (Q::kTwoWeights)
                        w.acc[4 * u + e][n] = QFp16::mfma(f[e], rest[q][n], w.acc[4 * u + e][n]);
                }
        }
}

// w with its NaN codes as zeros.
__device__ __forceinline__ uint32_t without_nans(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xffu); }

// Clears the value codes of keys that are not there (bits of ok); whether a
// NaN code is left.
template <int D>
__device__ __forceinline__ bool clear_hidden(Raw<D>& raw, uint32_t ok) {
    uint32_t any_nan = 0;
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            raw.v[u][j] = ok >> j & 1 ? raw.v[u][j] : 0u;
            any_nan |= nan_codes(raw.v[u][j]);
        }
    return __any(any_nan != 0);
}

// What a wave works on.
struct Task {
    int b, kvh;
    int t;                             // the query, with indices
    int row0, rows;                    // first row of the wave, rows of the group
    int part;
    bool live;
};

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

}  // namespace lix
