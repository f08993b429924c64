// Softmax attention over the 8-bit cache (lix_kv8_attention): many rows.
//
// A workgroup's W waves own 16 NT rows each and pass over the same keys, KT at
// a time (kv8_rows.h).  Their codes are loaded and converted once for the
// workgroup, into operand fragments in LDS: a fragment is 64 lanes x 16 bytes
// in lane order, so it is written and read without bank conflicts.  Two
// buffers: the codes of the next tile are on their way from memory while the
// present one is used, and are converted into the other buffer before the one
// barrier of a tile.
#include <hip/hip_runtime.h>

#include "kv8_rows.h"

namespace lix {

namespace {

template <int D, int KT>
struct Tile {
    u32x4 k[KT / 16][D / 32][64];
    u32x4 v[KT / 32][D / 16][64];
};

// Fragments of a tile's keys from LDS.
template <class Q, int D, int KT>
struct SharedKeys {
    static constexpr bool kShared = true;
    const Tile<D, KT>& t;
    int first;                         // 16-key tile it starts at
    int lane;
    __device__ __forceinline__ typename Q::frag key(int h, int ks) const {
        return __builtin_bit_cast(typename Q::frag, t.k[first + h][ks][lane]);
    }
    __device__ __forceinline__ void values(int q, int u, f16x8 (&f)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __builtin_bit_cast(f16x8, t.v[first / 2 + q][4 * u + e][lane]);
    }
};

// A wave's share of a tile: units of 16 keys' codes (all dimensions) or of 32
// values' codes (one 4-byte group of each lane), one after another.
template <int D, int KT, int W>
struct Share {
    static constexpr int KU = KT / 16, VU = KT / 32 * (D / 64);
    static constexpr int N = (KU + VU + W - 1) / W;
    static constexpr int WORDS = D / 16 > 8 ? D / 16 : 8;
    uint32_t w[N][WORDS];
};

template <int D, int WORDS>
__device__ __forceinline__ void load_key_unit(uint32_t (&w)[WORDS], const uint8_t* __restrict__ p) {
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(p + 64 * u);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * u + i] = x[i];
    }
}

template <class Q, int D, int KT, int W>
__device__ __forceinline__ void store_unit(Tile<D, KT>& t, const Share<D, KT, W>& s, int i, int unit, int lane) {
    using S = Share<D, KT, W>;
    if (unit < S::KU) {
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks)
            t.k[unit][ks][lane] = __builtin_bit_cast(u32x4, key_frag<Q>(s.w[i][2 * ks], s.w[i][2 * ks + 1]));
    } else if (unit < S::KU + S::VU) {
        const int x = unit - S::KU, p = x / (D / 64), u = x % (D / 64);
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = s.w[i][j];
        f16x8 f[4];
        value_frags(v, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) t.v[p][4 * u + e][lane] = __builtin_bit_cast(u32x4, f[e]);
    }
}

// Clears the value codes of a unit's hidden keys (bits j of ok: key 16 (j / 4)
// + 4 g + j % 4 of the 32 is there) and, with NANS, its NaN codes; whether
// there were any.
template <bool NANS, int WORDS>
__device__ __forceinline__ bool clear_unit(uint32_t (&w)[WORDS], uint32_t ok) {
    uint32_t bad = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        w[j] = ok >> j & 1 ? w[j] : 0u;
        bad |= nan_codes(w[j]);
        if (NANS) w[j] = without_nans(w[j]);
    }
    return __any(bad != 0);
}

// The workgroup's task, with the wave's own first row.
template <int NT, int W, bool SEL>
__device__ __forceinline__ Task group_task(const AttendArgs& a, const AttendPlan& plan, int wave) {
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
    int group;
    if (SEL) {
        group = (int)(u % plan.row_tiles);
        k.t = (int)(u / plan.row_tiles);
        k.rows = a.q.G;
    } else {
        group = plan.row_tiles - 1 - (int)u;       // late rows see the most keys: they go first
        k.t = 0;
        k.rows = a.q.S * a.q.G;
    }
    k.row0 = (group * W + wave) * 16 * NT;
    return k;
}

// ---------------------------------------------------------------- all visible tokens

// Tokens come in entries of 16 (a page holds whole entries).  Lane e of every
// wave looks up entry e of the next 64: row of the cache and scales, which are
// then read from that lane when their tile's turn comes.  The lookups of the
// next 64 entries run while the present ones are used.
template <class Q, int D, int NT, int W, int KT>
__global__ __launch_bounds__(64 * W, 2) void kv8_dense_tiles_kernel(AttendArgs a, AttendPlan plan) {
    using S = Share<D, KT, W>;
    constexpr int E = KT / 16, kBatch = 64 / E;    // entries of a tile, tiles of a batch
    __shared__ Tile<D, KT> tiles[2];
    __shared__ int nan_at[2][W];       // NaN among the values that a wave put into the tile
    __shared__ int range[2][W];        // most and least visible keys of each wave's rows
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Task k = group_task<NT, W, false>(a, plan, wave);
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int shift = a.c.page_shift;
    const int len = cached_len(a.c, k.b);
    const bool has_rows = k.row0 < k.rows;         // a wave behind the last row only helps to load

    // keys [0, most) are seen by some row of the wave, [0, least) by all; the
    // same for the workgroup
    int vis[NT];
    const int last = min(k.row0 + 16 * NT, k.rows) - 1;
    int most = 0, least = len;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = min(k.row0 + 16 * n + (lane & 15), last);
        vis[n] = has_rows ? visible_tokens(a.q, k.b, r / a.q.G, len) : 0;
        most = max(most, vis[n]);
        least = min(least, vis[n]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        most = max(most, __shfl_xor(most, o));
        least = min(least, __shfl_xor(least, o));
    }
    if (lane == 0) {
        range[0][wave] = most;
        range[1][wave] = has_rows ? least : len;
    }
    __syncthreads();
    int group_most = 0, group_least = len;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        group_most = max(group_most, range[0][i]);
        group_least = min(group_least, range[1][i]);
    }
    most = __builtin_amdgcn_readfirstlane(most);
    least = __builtin_amdgcn_readfirstlane(least);
    group_most = __builtin_amdgcn_readfirstlane(group_most);
    group_least = __builtin_amdgcn_readfirstlane(group_least);
    const int chunk = ((group_most + plan.parts - 1) / plan.parts + KT - 1) / KT * KT;
    const int lo = (int)min((long)k.part * chunk, (long)group_most);
    const int hi = (int)min((long)lo + chunk, (long)group_most);

    Rows<Q, D, NT> w;
    w.init();
    if (lo < hi) {
        if (has_rows) load_queries<Q, D, NT, false>(a, k, w);
        const int32_t* table = a.c.table + (long)k.b * a.c.max_pages;
        // the batch of the tile that is loaded: rows, which are there, scales
        int row = 0;
        uint64_t good = 0;
        float kscale = 0.0f, vscale = 0.0f;
        int token = lo + 16 * lane, pid = -1;      // of the batch behind it
        auto find = [&]() { pid = token < hi ? table[token >> shift] : -1; };
        auto look = [&]() {
            const bool there = pid >= 0 && pid < a.c.num_pages;
            const long at = (long)(there ? pid : 0) * a.c.Hkv + k.kvh;
            row = there ? (int)((at << shift) + (token & ((1 << shift) - 1))) : 0;
            kscale = there ? a.c.k_scale[at] : 0.0f;
            vscale = there ? a.c.v_scale[at] : 0.0f;
            good = __ballot(there);
            token = token < hi ? token + 1024 : token;
            find();
        };
        // the batch of the tile that is used
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

        S share;
        const uint32_t k_off = (lane & 15) * D + 16 * g, v_off = 4 * g * D + (lane & 15) * (D / 16);
        // codes of the tile whose first entry of the batch is e0
        auto load = [&](int e0) {
#pragma unroll
            for (int i = 0; i < S::N; ++i) {
                const int unit = wave + i * W;
                if (unit < S::KU) {
                    const long at = __builtin_amdgcn_readlane(row, e0 + unit);
                    load_key_unit<D>(share.w[i], a.c.k + at * D + k_off);
                } else if (unit < S::KU + S::VU) {
                    const int x = unit - S::KU, p = x / (D / 64), u = x % (D / 64);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const long at = __builtin_amdgcn_readlane(row, e0 + 2 * p + h);
                        const uint8_t* v = a.c.v + at * D + 4 * u;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            share.w[i][4 * h + j] = *reinterpret_cast<const uint32_t*>(v + v_off + (uint32_t)(j * D));
                    }
                }
            }
        };
        // converts them, the tile at s0, into buffer `to`
        auto store = [&](int s0, int e0, int to) {
            const uint32_t there = (uint32_t)(good >> e0) & ((1u << E) - 1);
            const bool edge = there != (1u << E) - 1 || s0 + KT > group_least || s0 + KT > hi;
            bool nans = false;
#pragma unroll
            for (int i = 0; i < S::N; ++i) {
                const int unit = wave + i * W;
                if (edge && unit >= S::KU && unit < S::KU + S::VU) {
                    const int p = (unit - S::KU) / (D / 64);
                    uint32_t ok = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        ok |= (there >> (2 * p + j / 4) & 1) && s0 + 32 * p + key_of(j, g) < hi ? 1u << j : 0u;
                    nans |= clear_unit<true>(share.w[i], ok);
                }
                store_unit<Q>(tiles[to], share, i, unit, lane);
            }
            if (edge && lane == 0) nan_at[to][wave] = nans;
        };

        find();
        look();
        load(0);
        store(lo, 0, 0);
        __syncthreads();
        int cur = 0, t = 0;            // t: the tile's place in its batch
        for (int s0 = lo; s0 < hi; s0 += KT) {
            if (t == 0) use();
            const bool more = s0 + KT < hi;
            const int next = t + 1 == kBatch ? 0 : t + 1;
            if (more) {
                if (next == 0) look();
                load(next * E);
            }
            if (has_rows && s0 < most) {
                const uint32_t there = (uint32_t)(used >> (t * E)) & ((1u << E) - 1);
                const bool edge = there != (1u << E) - 1 || s0 + KT > least || s0 + KT > hi;
                Scales<E, false> sc;
#pragma unroll
                for (int h = 0; h < E; ++h) {
                    auto lane_of = [&](float v) {
                        return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), t * E + h));
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
                    for (int j = 0; j < 4 * E; ++j)
                        ok |= (there >> (j / 4) & 1) && s0 + key_of(j, g) < hi ? 1u << j : 0u;
                }
                if (there != (1u << E) - 1 || s0 + KT > group_least || s0 + KT > hi) {
                    // an edge for some wave of the workgroup: NaN codes are out of it
                    bool nans = false;
#pragma unroll
                    for (int i = 0; i < W; ++i) nans |= nan_at[cur][i] != 0;
                    if (nans) {
                        auto codes = [&](int q, int u, uint32_t (&v)[8]) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int s = s0 + 32 * q + key_of(j, g);
                                const int pid = s < hi ? table[s >> shift] : -1;
                                const bool is = pid >= 0 && pid < a.c.num_pages;
                                const long at =
                                    (((long)(is ? pid : 0) * a.c.Hkv + k.kvh) << shift) + (s & ((1 << shift) - 1));
                                v[j] = is ? *reinterpret_cast<const uint32_t*>(a.c.v + at * D + (lane & 15) * (D / 16) +
                                                                               4 * u)
                                          : 0u;
                            }
                        };
                        mark_nans<Q, D, NT, E>(w, codes, left, ok);
                    }
                }
                step<Q, D, NT, E, false>(w, SharedKeys<Q, D, KT>{tiles[cur], 0, lane}, sc, edge, left, ok);
            }
            if (more) store(s0 + KT, next * E, cur ^ 1);
            __syncthreads();
            cur ^= 1;
            t = next;
        }
    }
    if (has_rows) store_rows<Q, D, NT, false>(a, plan, k, w);
}

// ---------------------------------------------------------------- given tokens

// What the waves need of 64 entries of an index list.
struct ListInfo {
    float c[64];                       // scale log2(e) k_scale
    float r[64];                       // v_scale / ref
    float ref;                         // bound of the v_scale up to these entries
    uint32_t ok[2];                    // entries that are there
};

// One query's list, 32 entries a tile, for four waves of 16 heads each: two load
// and convert the keys, the others the values, two tiles ahead of the one in use
// (a gather from L2 takes longer than a tile).  16 heads to a wave, not 32: the
// fragments are read from LDS twice as often, but four waves fit a SIMD instead
// of two and cover each other's trips to LDS (@@).  Lane e of all looks up entry e of the
// next 64: its token and page while the entries before are used, its row of the
// cache and scales when their codes are to be loaded, so that no load waits for
// another's address.  FAR: the pages pass 4 GiB, offsets into them take 64 bits.
template <class Q, int D, int NT, bool FAR>
__global__ __launch_bounds__(256, D <= 128 ? 4 : 2) void kv8_selected_tiles_kernel(AttendArgs a, AttendPlan plan) {
    constexpr int W = 4, KT = 32, VB = D / 16;     // VB: a lane's value codes of one key
    constexpr int VH = D <= 128 ? 1 : D / 128;     // 4-byte groups of them that a wave takes
    __shared__ Tile<D, KT> tiles[2];
    __shared__ ListInfo infos[2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Task k = group_task<NT, W, true>(a, plan, wave);
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int shift = a.c.page_shift;
    const int seen = __builtin_amdgcn_readfirstlane(visible_tokens(a.q, k.b, k.t, cached_len(a.c, k.b)));
    const bool has_rows = k.row0 < k.rows;         // a wave behind the last row only helps to load
    const int all = seen > 0 ? a.topk : 0;
    const int chunk = ((all + plan.parts - 1) / plan.parts + KT - 1) / KT * KT;
    const int lo = (int)min((long)k.part * chunk, (long)all), hi = (int)min((long)lo + chunk, (long)all);

    Rows<Q, D, NT> w;
    w.init();
    if (lo < hi) {
        if (has_rows) load_queries<Q, D, NT, true>(a, k, w);
        const int32_t* table = a.c.table + (long)k.b * a.c.max_pages;
        const int32_t* list = a.indices + ((long)k.b * a.q.S + k.t) * a.topk;
        // this lane's entry of the next 64: its token (the one behind: ahead), its page
        auto entry = [&](int e) {
            const int idx = e < hi ? list[e] : -1;
            return idx < seen ? idx : -1;
        };
        auto page_of = [&](int idx) { return idx >= 0 ? table[idx >> shift] : -1; };
        int at_entry = lo + lane;
        int idx = entry(at_entry), pid = page_of(idx), ahead = entry(at_entry + 64);
        // the 64 entries whose codes are loaded: byte offsets, scales, which are there
        uint32_t off = 0, off_hi = 0;
        float kscale = 0.0f, vscale = 0.0f;
        uint64_t good = 0;
        auto look = [&]() {
            const bool there = pid >= 0 && pid < a.c.num_pages;
            const long at = (long)(there ? pid : 0) * a.c.Hkv + k.kvh;
            const uint64_t byte = there ? (uint64_t)((at << shift) + (idx & ((1 << shift) - 1))) * D : 0;
            off = (uint32_t)byte;
            off_hi = (uint32_t)(byte >> 32);
            kscale = there ? a.c.k_scale[at] : 0.0f;
            vscale = there ? a.c.v_scale[at] : 0.0f;
            good = __ballot(there);
            idx = ahead;
            pid = page_of(idx);
            at_entry = at_entry < hi ? at_entry + 64 : at_entry;
            ahead = entry(at_entry + 64);
        };
        float ref = 0.0f;
        auto inform = [&](ListInfo& info) {
            float top = vscale;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
            if (top > ref) ref = top * kRefRoom;
            info.c[lane] = kscale * a.q.scale_log2;
            info.r[lane] = ref > 0.0f ? vscale * __builtin_amdgcn_rcpf(ref) : 0.0f;
            if (lane == 0) {
                info.ref = ref;
                info.ok[0] = (uint32_t)good;
                info.ok[1] = (uint32_t)(good >> 32);
            }
        };
        // address of dimension 0 of entry e
        auto row_at = [&](const uint8_t* base, int e, uint32_t more) {
            const uint32_t x = __builtin_amdgcn_ds_bpermute(4 * e, off) + (FAR ? 0 : more);
            if constexpr (FAR)
                return base + (((uint64_t)__builtin_amdgcn_ds_bpermute(4 * e, off_hi) << 32 | x) + more);
            else
                return base + x;
        };

        struct Codes {
            uint32_t w[VB > 8 * VH ? VB : 8 * VH];
        };
        const bool does_keys = wave < 2, does_values = !does_keys && (wave - 2) * VH < D / 64;
        auto load = [&](Codes& x, int e0) {        // e0: the tile's first of the 64 entries
            if (does_keys) {
                const uint8_t* p = row_at(a.c.k, e0 + 16 * wave + (lane & 15), 16 * g);
#pragma unroll
                for (int u = 0; u < D / 64; ++u) {
                    const u32x4 v = *reinterpret_cast<const u32x4*>(p + 64 * u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x.w[4 * u + i] = v[i];
                }
            } else if (does_values) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint8_t* p =
                        row_at(a.c.v, e0 + 4 * g + (16 * (j / 4) + j % 4), (lane & 15) * VB + 4 * VH * (wave - 2));
                    if constexpr (VH == 1) {
                        x.w[j] = *reinterpret_cast<const uint32_t*>(p);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(p);
                        x.w[j] = v.x;
                        x.w[8 + j] = v.y;
                    }
                }
            }
        };
        // converts them into buffer `to`; there: which of the tile's entries are
        auto store = [&](const Codes& x, uint32_t there, int to) {
            Tile<D, KT>& t = tiles[to];
            if (does_keys) {
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks)
                    t.k[wave][ks][lane] = __builtin_bit_cast(u32x4, key_frag<Q>(x.w[2 * ks], x.w[2 * ks + 1]));
            } else if (does_values) {
                uint32_t ok = ~0u;
                if (there != ~0u) {
                    ok = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ok |= (there >> key_of(j, g) & 1) << j;
                }
#pragma unroll
                for (int u = 0; u < VH; ++u) {
                    uint32_t v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = x.w[8 * u + j];
                    if (there != ~0u) clear_unit<false>(v, ok);
                    f16x8 f[4];
                    value_frags(v, f);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        t.v[0][4 * (VH * (wave - 2) + u) + e][lane] = __builtin_bit_cast(u32x4, f[e]);
                }
            }
        };
        auto compute = [&](int i) {                // tile i
            const ListInfo& info = infos[i >> 1 & 1];
            const float next_ref = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(info.ref)));
            if (next_ref > w.ref) w.set_ref(next_ref);
            const int e0 = 32 * (i & 1);
            Scales<2, true> sc;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 c4 = *reinterpret_cast<const f32x4*>(&info.c[e0 + 16 * h + 4 * g]);
                const f32x4 r4 = *reinterpret_cast<const f32x4*>(&info.r[e0 + 16 * h + 4 * g]);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    sc.c[4 * h + x] = c4[x];
                    sc.r[4 * h + x] = r4[x];
                }
            }
            const uint32_t there = __builtin_amdgcn_readfirstlane(info.ok[i & 1]);
            uint32_t ok = ~0u;
            if (there != ~0u) {
                ok = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) ok |= (there >> key_of(j, g) & 1) << j;
            }
            const int none[NT] = {};
            step<Q, D, NT, 2, true>(w, SharedKeys<Q, D, KT>{tiles[i & 1], 0, lane}, sc, there != ~0u, none, ok);
        };

        // Even tiles pass through `even`, odd ones through `odd`; tile i is used
        // from buffer i & 1.  held: the entries that are there of the 64 whose
        // tiles are stored, good: of those whose codes are loaded.
        const int count = (hi - lo + KT - 1) / KT;
        Codes even, odd;
        look();
        load(even, 0);
        if (count > 1) load(odd, 32);
        if (wave == 0) inform(infos[0]);
        uint64_t held = good;
        store(even, (uint32_t)held, 0);
        if (count > 2) {
            look();
            load(even, 0);
        }
        __syncthreads();
        for (int i = 0; i < count; i += 2) {
            if (has_rows) compute(i);
            if (i + 1 < count) store(odd, (uint32_t)(held >> 32), 1);
            if (i + 3 < count) load(odd, 32);
            __syncthreads();
            if (i + 1 >= count) break;
            if (has_rows) compute(i + 1);
            if (i + 2 < count) {
                if (wave == 0) inform(infos[(i + 2) >> 1 & 1]);
                held = good;
                store(even, (uint32_t)held, 0);
            }
            if (i + 4 < count) {
                look();
                load(even, 0);
            }
            __syncthreads();
        }
    }
    if (has_rows) store_rows<Q, D, NT, true>(a, plan, k, w);
}

template <class Q, int D>
hipError_t launch(const AttendArgs& a, const AttendPlan& plan) {
    const bool sel = a.indices != nullptr;
    const long grid = plan.tasks * plan.row_tiles * plan.parts;
    auto go = [&](auto kernel, int waves) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * waves), 0, a.stream, a, plan);
    };
    constexpr int KT = D <= 128 ? 64 : 32;
    constexpr int NT = D <= 128 ? 2 : 1;
    const bool far = ((double)a.c.num_pages * a.c.Hkv * D) * (1 << a.c.page_shift) > 4294967296.0;
    if (!sel && plan.waves == 8) go(kv8_dense_tiles_kernel<Q, D, NT, 8, KT>, 8);
    else if (!sel) go(kv8_dense_tiles_kernel<Q, D, NT, 4, KT>, 4);
    else far ? go(kv8_selected_tiles_kernel<Q, D, 1, true>, 4) : go(kv8_selected_tiles_kernel<Q, D, 1, false>, 4);
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

hipError_t launch_kv8_tiles(const AttendArgs& a, const AttendPlan& plan) {
    return a.q.dtype == LIX_BF16 ? launch_dim<QBf16>(a, plan) : launch_dim<QFp16>(a, plan);
}

}  // namespace lix
