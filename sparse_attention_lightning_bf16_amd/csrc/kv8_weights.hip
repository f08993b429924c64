// The attention weight that each cached token got (lix_kv8_token_weights):
//     w[s] = sum over the rows (queries x heads of a key head) that see s of
//            2^(scale log2(e) k_scale (q . code[s]) - log2(e) lse)
//
// Keys are the rows of the product (kv8_core.h): a lane adds up its own keys
// over all rows that pass, and the sum over the 16 row columns is taken once,
// at the end.  No atomics, the same order on every call.
//
// Many rows: a wave keeps 64 keys (32 for D = 256) as operand fragments in
// registers, and the four waves of a workgroup, with neighbouring keys, pass over
// the same rows, 64 at a time: each brings 16 of them into LDS as fragments, the
// next while the present ones are used (without LDS the waves' reads of the same
// rows were bound by L1).  The rows of a key range are split into parts where
// there are too few ranges; their sums go to the workspace and are added by a
// second kernel.  Bound by the exponentials and the products.
//
// One tile of 16 rows: the rows stay in registers and the keys pass by, 16 at
// a time per step and two steps ahead, 64 steps' pages looked up at once.  Bound
// by reading the key codes.
#include <hip/hip_runtime.h>

#include "kv8_core.h"

namespace lix {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// v summed over the 16 lanes of a row group (l % 16), in every lane.
__device__ __forceinline__ float row_sum(float v) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xf, 0xf, true));      // row_ror:8
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xf, 0xf, true));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xf, 0xf, true));
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x121, 0xf, 0xf, true));
}

// ---------------------------------------------------------------- many rows

template <class Q, int D, int KT>
__global__ __launch_bounds__(256, 2) void kv8_weights_kernel(WeighArgs a) {
    constexpr int KS = D / 32;
    __shared__ u32x4 stage[2][4][KS][64];          // [buffer][16-row tile][step][lane]
    __shared__ float stage_lse[2][64];
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long pairs = (long)a.q.B * a.c.Hkv;
    const long pair = blockIdx.x % pairs;
    long u = blockIdx.x / pairs;
    const int part = (int)(u % a.parts);
    u /= a.parts;
    const int b = (int)(pair / a.c.Hkv), kvh = (int)(pair % a.c.Hkv);
    const int len = cached_len(a.c, b);
    const long g_first = u * 4 * (16L * KT);       // the workgroup's first key
    if (g_first >= len) return;
    const int s0 = (int)min(g_first + wave * 16 * KT, (long)len);      // a wave behind the end only brings rows
    const int shift = a.c.page_shift;

    typename Q::frag key[KT][KS];
    float c[KT];
    bool exists[KT];
#pragma unroll
    for (int h = 0; h < KT; ++h) {
        const int s = s0 / 16 * 16 + 16 * h;
        const int nth = s >> shift;
        int pid = nth < a.c.max_pages ? a.c.table[(long)b * a.c.max_pages + nth] : -1;
        exists[h] = s < len && pid >= 0 && pid < a.c.num_pages;
        pid = exists[h] ? pid : 0;
        const long at = (long)pid * a.c.Hkv + kvh;
        const uint8_t* p = a.c.k + ((at << shift) + (s & ((1 << shift) - 1)) + (lane & 15)) * D + 16 * g;
        c[h] = exists[h] ? a.c.k_scale[at] * a.q.scale_log2 : 0.0f;
#pragma unroll
        for (int u4 = 0; u4 < D / 64; ++u4) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(p + 64 * u4);
            key[h][2 * u4] = key_frag<Q>(w[0], w[1]);
            key[h][2 * u4 + 1] = key_frag<Q>(w[2], w[3]);
        }
    }

    // Rows [first, all_from) see some of the wave's keys, [all_from, rows) all of
    // them; rows behind the last query are left out.  The workgroup starts at the
    // first row that sees any of its keys.
    const int G = a.q.G;
    const int queries = a.q.q_lens ? min(max(a.q.q_lens[b], 0), a.q.S) : a.q.S;
    const int rows = queries * G;
    auto sees = [&](long s) {                      // first row that sees token s
        if (a.q.q_start == nullptr) return 0;
        return (int)min(max((s + 1) * a.q.ratio - 1 - a.q.q_start[b], 0L), (long)queries) * G;
    };
    const int g_row = sees(g_first), first = s0 < len ? sees(s0) : rows;
    const int all_from = s0 + 16 * KT > len ? rows : sees((long)s0 + 16 * KT - 1);
    const int tiles = (rows - g_row + 15) / 16;
    const int per_part = ((tiles + a.parts - 1) / a.parts + 3) / 4 * 4;
    const int t_lo = min(part * per_part, tiles), t_hi = min(t_lo + per_part, tiles);

    f32x4 sum[KT];
#pragma unroll
    for (int h = 0; h < KT; ++h) sum[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (t_lo < t_hi) {
        const typename Q::elem* q = static_cast<const typename Q::elem*>(a.q.q) + b * a.q.sb + 16 * g;
        // query and head of this lane's row of the wave's next tile
        const int r_first = g_row + 16 * (t_lo + wave) + (lane & 15);
        int t = r_first / G, h_of = r_first - t * G;
        const int step_t = 64 / G, step_h = 64 - step_t * G;
        typename Q::frag held[KS];
        float held_lse = 0.0f;
        auto load = [&]() {
            const bool in = t < queries;
            const int tt = in ? t : queries - 1, head = kvh * G + (in ? h_of : 0);
            const typename Q::elem* at = q + tt * a.q.ss + head * a.q.sh;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                held[ks] = *reinterpret_cast<const typename Q::frag*>(at + 64 * (ks / 2) + 8 * (ks & 1));
            held_lse = a.lse[((long)b * a.q.S + tt) * a.q.Hq + head];
            t += step_t;
            h_of += step_h;
            const bool wrap = h_of >= G;
            t += wrap ? 1 : 0;
            h_of -= wrap ? G : 0;
        };
        auto store = [&](int to) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) stage[to][wave][ks][lane] = __builtin_bit_cast(u32x4, held[ks]);
            if (lane < 16) stage_lse[to][16 * wave + lane] = held_lse;
        };
        auto add = [&](int from, int x, int i) {   // tile i, the x-th of the buffer
            const int r0 = g_row + 16 * i;
            if (r0 + 16 <= first) return;
            typename Q::frag f[KS];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) f[ks] = __builtin_bit_cast(typename Q::frag, stage[from][x][ks][lane]);
            const float lse = stage_lse[from][16 * x + (lane & 15)];
            // a row whose lse is -inf gives nothing, whatever its scores are
            const bool edge = r0 < all_from || r0 + 16 > rows || __any(lse == neg_inf());
            const float base = -lse * kLog2e;
            int vis = 0;
            if (edge) {
                const int r = r0 + (lane & 15);
                vis = r < rows && lse != neg_inf() ? visible_tokens(a.q, b, r / G, len) - s0 : 0;
            }
#pragma unroll
            for (int h = 0; h < KT; ++h) {
                f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) y = Q::mfma(key[h][ks], f[ks], y);
                f32x4 p;
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(y[j], c[h], base));
                if (edge) {
                    int here = 4 * g;
                    asm volatile("" : "+v"(here));              // the masks stay inside the branch
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = 16 * h + here + j < vis ? p[j] : 0.0f;
                }
                sum[h] += p;
            }
        };
        load();
        store(0);
        __syncthreads();
        int cur = 0;
        for (int i = t_lo; i < t_hi; i += 4) {
            if (i + 4 < t_hi) load();
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (i + x < t_hi) add(cur, x, i + x);
            if (i + 4 < t_hi) store(cur ^ 1);
            __syncthreads();
            cur ^= 1;
        }
    }
#pragma unroll
    for (int h = 0; h < KT; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = exists[h] ? row_sum(sum[h][i]) : 0.0f;
            const int s = s0 + 16 * h + 4 * g + i;
            if ((lane & 15) != i || s >= len) continue;
            if (a.parts > 1) {
                a.workspace[(part * pairs + pair) * a.cap + s] = v;
            } else {
                float* w = a.weights + pair * a.width + s;
                *w = a.accumulate ? *w + v : v;
            }
        }
}

// The parts' sums of each token, in order.
__global__ __launch_bounds__(256) void kv8_weights_join_kernel(WeighArgs a) {
    const long pairs = (long)a.q.B * a.c.Hkv;
    const long pair = blockIdx.x % pairs;
    const int s = (int)(blockIdx.x / pairs) * 256 + threadIdx.x;
    if (s >= cached_len(a.c, (int)(pair / a.c.Hkv))) return;
    float v = 0.0f;
    for (int p = 0; p < a.parts; ++p) v += a.workspace[(p * pairs + pair) * a.cap + s];
    float* w = a.weights + pair * a.width + s;
    *w = a.accumulate ? *w + v : v;
}

// ---------------------------------------------------------------- one tile of rows


template <class Q, int D>
__global__ __launch_bounds__(256, 2) void kv8_weights_few_kernel(WeighArgs a, int range) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long pairs = (long)a.q.B * a.c.Hkv;
    const long pair = blockIdx.x % pairs;
    const int b = (int)(pair / a.c.Hkv), kvh = (int)(pair % a.c.Hkv);
    const int len = cached_len(a.c, b);
    const long first = (blockIdx.x / pairs * 4 + wave) * (long)range;
    if (first >= len) return;
    const int lo = (int)first, hi = min(lo + range, len);
    const int shift = a.c.page_shift, G = a.q.G, rows = a.q.S * G;

    // lane e: entry e of 16 keys, its row of the cache and scale
    const int token = lo + 16 * lane;
    const int pid = token < hi ? a.c.table[(long)b * a.c.max_pages + (token >> shift)] : -1;
    const bool there = pid >= 0 && pid < a.c.num_pages;
    const long at = (long)(there ? pid : 0) * a.c.Hkv + kvh;
    const int row = there ? (int)((at << shift) + (token & ((1 << shift) - 1))) : 0;
    const float scale = there ? a.c.k_scale[at] * a.q.scale_log2 : 0.0f;
    const uint64_t good = __ballot(there);

    const int r = lane & 15, rc = min(r, rows - 1);
    const int t = rc / G, head = kvh * G + rc - t * G;
    const typename Q::elem* q =
        static_cast<const typename Q::elem*>(a.q.q) + b * a.q.sb + t * a.q.ss + head * a.q.sh + 16 * g;
    typename Q::frag f[D / 32];
    const uint32_t off = (lane & 15) * D + 16 * g;
    struct Codes {
        u32x4 w[2][D / 64];
    };
    auto load = [&](Codes& x, int i) {             // keys 32 i .. of the range
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t* p = a.c.k + (long)__builtin_amdgcn_readlane(row, 2 * i + h) * D;
#pragma unroll
            for (int u = 0; u < D / 64; ++u) x.w[h][u] = *reinterpret_cast<const u32x4*>(p + (off + 64u * u));
        }
    };
    const int steps = (hi - lo + 31) / 32;
    Codes one, two;
    load(one, 0);
    if (steps > 1) load(two, 1);
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks) f[ks] = *reinterpret_cast<const typename Q::frag*>(q + 64 * (ks / 2) + 8 * (ks & 1));
    const float lse = a.lse[((long)b * a.q.S + t) * a.q.Hq + head];
    const int vis = r < rows && lse != neg_inf() ? visible_tokens(a.q, b, t, len) : 0;
    const float base = -lse * kLog2e;
    int least = vis;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) least = min(least, __shfl_xor(least, o));
    least = __builtin_amdgcn_readfirstlane(least);

    float* w = a.weights + pair * a.width;
    auto add = [&](const Codes& x, int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int s0 = lo + 32 * i + 16 * h;
            const float c = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale), 2 * i + h));
            f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                y = Q::mfma(key_frag<Q>(x.w[h][u][0], x.w[h][u][1]), f[2 * u], y);
                y = Q::mfma(key_frag<Q>(x.w[h][u][2], x.w[h][u][3]), f[2 * u + 1], y);
            }
            f32x4 p;
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(y[j], c, base));
            if (s0 + 16 > least) {
                const bool is = good >> (2 * i + h) & 1;
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = is && s0 + 4 * g + j < vis ? p[j] : 0.0f;
            } else if (!(good >> (2 * i + h) & 1)) {
                p = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = row_sum(p[j]);
            const int s = s0 + 4 * g + (lane & 3);
            const float v = lane & 2 ? (lane & 1 ? p[3] : p[2]) : (lane & 1 ? p[1] : p[0]);
            if ((lane & 15) < 4 && s < hi) w[s] = a.accumulate ? w[s] + v : v;
        }
    };
    for (int i = 0; i < steps; i += 2) {
        add(one, i);
        if (i + 2 < steps) load(one, i + 2);
        if (i + 1 < steps) add(two, i + 1);
        if (i + 3 < steps) load(two, i + 3);
    }
}

template <class Q, int D>
hipError_t launch(const WeighArgs& a, const WeighPlan& plan) {
    const long pairs = (long)a.q.B * a.c.Hkv;
    auto groups = [&](long keys) { return dim3((unsigned)(pairs * ((a.cap + 4 * keys - 1) / (4 * keys)) * plan.parts)); };
    if (plan.range > 0) {
        hipLaunchKernelGGL((kv8_weights_few_kernel<Q, D>), groups(plan.range), dim3(256), 0, a.stream, a, plan.range);
        return hipGetLastError();
    }
    constexpr int KT = D <= 128 ? 4 : 2;
    hipLaunchKernelGGL((kv8_weights_kernel<Q, D, KT>), groups(16 * KT), dim3(256), 0, a.stream, a);
    if (plan.parts > 1)
        hipLaunchKernelGGL(kv8_weights_join_kernel, dim3((unsigned)(pairs * ((a.cap + 255) / 256))), dim3(256), 0,
                           a.stream, a);
    return hipGetLastError();
}

template <class Q>
hipError_t launch_dim(const WeighArgs& a, const WeighPlan& plan) {
    switch (a.c.D) {
        case 64: return launch<Q, 64>(a, plan);
        case 128: return launch<Q, 128>(a, plan);
        default: return launch<Q, 256>(a, plan);
    }
}

}  // namespace

hipError_t launch_kv8_token_weights(const WeighArgs& a, const WeighPlan& plan) {
    return a.q.dtype == LIX_BF16 ? launch_dim<QBf16>(a, plan) : launch_dim<QFp16>(a, plan);
}

}  // namespace lix
