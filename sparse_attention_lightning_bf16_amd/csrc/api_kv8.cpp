// C ABI of the 8-bit cache (lix_kv8.h): validation and dispatch, on the host
// before any launch as in api.cpp.
#include <math.h>

#include "launch_kv8.h"
#include "lix_kv8.h"
#include "validate.h"

namespace {

using namespace lix;

int page_shift(int page) {
    switch (page) {
        case 16: return 4;
        case 32: return 5;
        case 64: return 6;
        case 128: return 7;
        default: return -1;
    }
}

// Sizes of the cache and its table.
int check_cache(int num_pages, int page, int Hkv, int D, int B, int max_pages) {
    if (num_pages <= 0 || page <= 0 || Hkv <= 0 || D <= 0 || B <= 0 || max_pages <= 0) return LIX_ERR_SHAPE;
    if (page_shift(page) < 0 || (D != 64 && D != 128 && D != 256)) return LIX_ERR_UNSUPPORTED;
    if ((long long)num_pages * Hkv >= (1LL << 31) / page) return LIX_ERR_UNSUPPORTED;
    if ((long long)max_pages * page >= (1LL << 30) || !fits(B, max_pages) || !fits(B, Hkv)) return LIX_ERR_UNSUPPORTED;
    return LIX_OK;
}

// Strides of 16-byte rows; those of dimensions of size one reach no address.
int check_strides(long long sb, int B, long long ss, int S, long long sh, int H) {
    const long long lim = 1LL << 40;
    const long long s[3] = {sb, ss, sh};
    const int n[3] = {B, S, H};
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < 0) return LIX_ERR_SHAPE;
        if (s[i] % 8 != 0 || s[i] > lim / n[i]) return LIX_ERR_UNSUPPORTED;
    }
    return LIX_OK;
}

int check_queries(int dtype, int B, int S, int Hq, int Hkv, int D, int ratio, float scale) {
    if (B <= 0 || S <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv != 0 || ratio < 1 || !(scale >= 0.0f) || !isfinite(scale))
        return LIX_ERR_SHAPE;
    if (dtype != LIX_BF16 && dtype != LIX_FP16) return LIX_ERR_SHAPE;
    if (!fits(B, S, Hq, D) || (long long)B * S * Hq > (1LL << 30)) return LIX_ERR_UNSUPPORTED;
    return LIX_OK;
}

// Grids are one-dimensional: their workgroups must fit 2^31.
bool grid_fits(double workgroups) { return workgroups < 2147483648.0; }

long zero_if(bool one, long long s) { return one ? 0 : (long)s; }

KV8Pages pages_of(const void* k, const void* v, const float* ks, const float* vs, int num_pages, int page, int Hkv,
                  int D, const int32_t* table, int max_pages, const int32_t* lens) {
    KV8Pages c{};
    c.k = static_cast<uint8_t*>(const_cast<void*>(k));
    c.v = static_cast<uint8_t*>(const_cast<void*>(v));
    c.k_scale = const_cast<float*>(ks);
    c.v_scale = const_cast<float*>(vs);
    c.num_pages = num_pages;
    c.page_shift = page_shift(page);
    c.Hkv = Hkv;
    c.D = D;
    c.table = table;
    c.max_pages = max_pages;
    c.lens = lens;
    return c;
}

QueryArgs queries_of(const void* q, long long sb, long long ss, long long sh, int dtype, int B, int S, int Hq, int Hkv,
                     const int32_t* q_start, const int32_t* q_lens, int ratio, float scale) {
    return QueryArgs{q, zero_if(B == 1, sb), zero_if(S == 1, ss), zero_if(Hq == 1, sh), dtype, B, S, Hq, Hq / Hkv,
                     q_start, q_lens, ratio, scale * 1.44269504088896340736f};
}

}  // namespace

extern "C" {

int lix_kv8_append(const void* k, long long k_sb, long long k_ss, long long k_sh, const void* v, long long v_sb,
                   long long v_ss, long long v_sh, int dtype, int B, int S, int Hkv, int D, void* k_pages,
                   void* v_pages, float* k_scales, float* v_scales, int num_pages, int page,
                   const int32_t* block_table, int max_pages, const int32_t* kv_lens, const int32_t* new_lens,
                   hipStream_t stream) {
    if (!k || !v || !k_pages || !v_pages || !k_scales || !v_scales || !block_table || !kv_lens) return LIX_ERR_NULL;
    if (S <= 0 || (dtype != LIX_BF16 && dtype != LIX_FP16)) return LIX_ERR_SHAPE;
    int st = check_cache(num_pages, page, Hkv, D, B, max_pages);
    if (st == LIX_OK) st = check_strides(k_sb, B, k_ss, S, k_sh, Hkv);
    if (st == LIX_OK) st = check_strides(v_sb, B, v_ss, S, v_sh, Hkv);
    if (st != LIX_OK) return st;
    if (!fits(B, S, Hkv, D) || S > (1 << 30) || !grid_fits((double)B * Hkv * 2 * ((S + page - 1) / page + 1)))
        return LIX_ERR_UNSUPPORTED;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
        !aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(block_table, 4) || !aligned(kv_lens, 4) ||
        !aligned(new_lens, 4))
        return LIX_ERR_UNSUPPORTED;
    st = check_device({k, v, k_pages, v_pages, k_scales, v_scales, block_table, kv_lens, new_lens});
    if (st != LIX_OK) return st;
    AppendArgs a{};
    a.x[0] = k;
    a.x[1] = v;
    a.sb[0] = zero_if(B == 1, k_sb);
    a.sb[1] = zero_if(B == 1, v_sb);
    a.ss[0] = zero_if(S == 1, k_ss);
    a.ss[1] = zero_if(S == 1, v_ss);
    a.sh[0] = zero_if(Hkv == 1, k_sh);
    a.sh[1] = zero_if(Hkv == 1, v_sh);
    a.dtype = dtype;
    a.B = B;
    a.S = S;
    a.c = pages_of(k_pages, v_pages, k_scales, v_scales, num_pages, page, Hkv, D, block_table, max_pages, kv_lens);
    a.new_lens = new_lens;
    a.stream = stream;
    return launch_status(launch_kv8_append(a));
}

long long lix_kv8_attention_workspace_bytes(int B, int S, int Hq, int Hkv, int D, int page, int max_pages, int topk) {
    if (topk < 0 || check_cache(1, page, Hkv, D, B, max_pages) != LIX_OK ||
        check_queries(LIX_BF16, B, S, Hq, Hkv, D, 1, 1.0f) != LIX_OK || (topk > 0 && !fits(B, S, topk)))
        return -1;
    return attend_plan(B, S, Hq, Hkv, D, page, max_pages, topk).workspace_bytes;
}

int lix_kv8_attention(const void* q, long long q_sb, long long q_ss, long long q_sh, int dtype, int B, int S, int Hq,
                      int Hkv, int D, const void* k_pages, const void* v_pages, const float* k_scales,
                      const float* v_scales, int num_pages, int page, const int32_t* block_table, int max_pages,
                      const int32_t* kv_lens, const int32_t* q_start, const int32_t* q_lens, int compress_ratio,
                      float scale, const int32_t* indices, int topk, void* out, float* lse, void* workspace,
                      long long workspace_bytes, hipStream_t stream) {
    if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !block_table || !kv_lens || !out || !lse)
        return LIX_ERR_NULL;
    int st = check_queries(dtype, B, S, Hq, Hkv, D, compress_ratio, scale);
    if (st != LIX_OK) return st;
    if (indices != nullptr && topk < 1) return LIX_ERR_SHAPE;
    st = check_cache(num_pages, page, Hkv, D, B, max_pages);
    if (st == LIX_OK) st = check_strides(q_sb, B, q_ss, S, q_sh, Hq);
    if (st != LIX_OK) return st;
    const int listed = indices != nullptr ? topk : 0;
    if (listed > 0 && (!fits(B, S, topk) || topk > (1 << 30))) return LIX_ERR_UNSUPPORTED;
    const AttendPlan plan = attend_plan(B, S, Hq, Hkv, D, page, max_pages, listed);
    if (!grid_fits((double)plan.tasks * plan.row_tiles * plan.parts)) return LIX_ERR_UNSUPPORTED;
    if (plan.workspace_bytes > 0 && workspace == nullptr) return LIX_ERR_NULL;
    if (workspace_bytes < plan.workspace_bytes) return LIX_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_scales, 4) ||
        !aligned(v_scales, 4) || !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(q_start, 4) ||
        !aligned(q_lens, 4) || !aligned(indices, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(workspace, 256))
        return LIX_ERR_UNSUPPORTED;
    st = check_device({q, k_pages, v_pages, k_scales, v_scales, block_table, kv_lens, q_start, q_lens, indices, out,
                       lse, plan.workspace_bytes > 0 ? workspace : nullptr});
    if (st != LIX_OK) return st;
    AttendArgs a{};
    a.q = queries_of(q, q_sb, q_ss, q_sh, dtype, B, S, Hq, Hkv, q_start, q_lens, compress_ratio, scale);
    a.c = pages_of(k_pages, v_pages, k_scales, v_scales, num_pages, page, Hkv, D, block_table, max_pages, kv_lens);
    a.indices = indices;
    a.topk = listed;
    a.out = out;
    a.lse = lse;
    a.workspace = static_cast<float*>(workspace);
    a.stream = stream;
    return launch_status(launch_kv8_attention(a, plan));
}

int lix_kv8_token_weights(const void* q, long long q_sb, long long q_ss, long long q_sh, int dtype, int B, int S,
                          int Hq, int Hkv, int D, const void* k_pages, const float* k_scales, int num_pages, int page,
                          const int32_t* block_table, int max_pages, const int32_t* kv_lens, const int32_t* q_start,
                          const int32_t* q_lens, int compress_ratio, float scale, const float* lse, float* weights,
                          int width, int accumulate, void* workspace, long long workspace_bytes,
                          hipStream_t stream) {
    if (!q || !k_pages || !k_scales || !block_table || !kv_lens || !lse || !weights) return LIX_ERR_NULL;
    int st = check_queries(dtype, B, S, Hq, Hkv, D, compress_ratio, scale);
    if (st == LIX_OK) st = check_cache(num_pages, page, Hkv, D, B, max_pages);
    if (st == LIX_OK) st = check_strides(q_sb, B, q_ss, S, q_sh, Hq);
    if (st != LIX_OK) return st;
    if (width < (long long)max_pages * page) return LIX_ERR_SHAPE;
    const WeighPlan plan = weigh_plan(B, S, Hq, Hkv, D, page, max_pages);
    if (!fits(B, Hkv, width) || !grid_fits((double)B * Hkv * max_pages * plan.parts)) return LIX_ERR_UNSUPPORTED;
    if (plan.workspace_bytes > 0 && workspace == nullptr) return LIX_ERR_NULL;
    if (workspace_bytes < plan.workspace_bytes) return LIX_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(k_scales, 4) || !aligned(block_table, 4) ||
        !aligned(kv_lens, 4) || !aligned(q_start, 4) || !aligned(q_lens, 4) || !aligned(lse, 4) || !aligned(weights, 4) ||
        !aligned(workspace, 256))
        return LIX_ERR_UNSUPPORTED;
    st = check_device({q, k_pages, k_scales, block_table, kv_lens, q_start, q_lens, lse, weights,
                       plan.workspace_bytes > 0 ? workspace : nullptr});
    if (st != LIX_OK) return st;
    WeighArgs a{};
    a.q = queries_of(q, q_sb, q_ss, q_sh, dtype, B, S, Hq, Hkv, q_start, q_lens, compress_ratio, scale);
    a.c = pages_of(k_pages, nullptr, k_scales, nullptr, num_pages, page, Hkv, D, block_table, max_pages, kv_lens);
    a.lse = lse;
    a.weights = weights;
    a.width = width;
    a.accumulate = accumulate;
    a.cap = (long)max_pages * page;
    a.parts = plan.parts;
    a.workspace = static_cast<float*>(workspace);
    a.stream = stream;
    return launch_status(launch_kv8_token_weights(a, plan));
}

long long lix_kv8_token_weights_workspace_bytes(int B, int S, int Hq, int Hkv, int D, int page, int max_pages) {
    if (check_cache(1, page, Hkv, D, B, max_pages) != LIX_OK ||
        check_queries(LIX_BF16, B, S, Hq, Hkv, D, 1, 1.0f) != LIX_OK)
        return -1;
    return weigh_plan(B, S, Hq, Hkv, D, page, max_pages).workspace_bytes;
}

long long lix_kv8_evict_workspace_bytes(int B, int Hkv, int page, int max_pages, int width, int keep, int recent,
                                        int sinks) {
    if (check_cache(1, page, Hkv, 64, B, max_pages) != LIX_OK || width <= 0 || keep <= 0 || recent < 0 || sinks < 0 || recent > keep ||
        sinks > keep - recent || !fits(B, Hkv, width) || !fits(B, Hkv, keep) || (long long)B * Hkv > (1LL << 30))
        return -1;
    return evict_layout(B, Hkv, (long)max_pages * page, width, keep, recent, sinks).total;
}

int lix_kv8_evict(void* k_pages, void* v_pages, float* k_scales, float* v_scales, int num_pages, int page, int B,
                  int Hkv, int D, const int32_t* block_table, int max_pages, const int32_t* kv_lens,
                  const float* weights, int width, const int32_t* new_table, int new_max_pages, int keep, int recent,
                  int sinks, int32_t* new_lens, int32_t* kept, float* new_weights, void* workspace,
                  long long workspace_bytes, hipStream_t stream) {
    if (!k_pages || !v_pages || !k_scales || !v_scales || !block_table || !kv_lens || !weights || !new_table ||
        !new_lens || !kept || !new_weights)
        return LIX_ERR_NULL;
    int st = check_cache(num_pages, page, Hkv, D, B, max_pages);
    if (st != LIX_OK) return st;
    if (width <= 0 || keep <= 0 || recent < 0 || sinks < 0 || recent > keep || sinks > keep - recent ||
        new_max_pages <= 0 || width < (long long)max_pages * page || (long long)new_max_pages * page < keep)
        return LIX_ERR_SHAPE;
    if (!fits(B, Hkv, width) || !fits(B, Hkv, keep) || !fits(B, new_max_pages) || (long long)B * Hkv > (1LL << 30) ||
        keep > (1 << 30) || !grid_fits((double)B * Hkv * 2 * ((keep + page - 1) / page)))
        return LIX_ERR_UNSUPPORTED;
    const EvictLayout ly = evict_layout(B, Hkv, (long)max_pages * page, width, keep, recent, sinks);
    if (ly.total > 0 && workspace == nullptr) return LIX_ERR_NULL;
    if (workspace_bytes < ly.total) return LIX_ERR_SHAPE;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_scales, 4) || !aligned(v_scales, 4) ||
        !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(weights, 4) || !aligned(new_table, 4) ||
        !aligned(new_lens, 4) || !aligned(kept, 4) || !aligned(new_weights, 4) || !aligned(workspace, 256))
        return LIX_ERR_UNSUPPORTED;
    st = check_device({k_pages, v_pages, k_scales, v_scales, block_table, kv_lens, weights, new_table, new_lens, kept,
                       new_weights, ly.total > 0 ? workspace : nullptr});
    if (st != LIX_OK) return st;
    EvictArgs a{};
    a.c = pages_of(k_pages, v_pages, k_scales, v_scales, num_pages, page, Hkv, D, block_table, max_pages, kv_lens);
    a.B = B;
    a.weights = weights;
    a.width = width;
    a.new_table = new_table;
    a.new_max_pages = new_max_pages;
    a.keep = keep;
    a.recent = recent;
    a.sinks = sinks;
    a.new_lens = new_lens;
    a.kept = kept;
    a.new_weights = new_weights;
    a.workspace = workspace;
    a.stream = stream;
    return launch_status(launch_kv8_evict(a, ly));
}

}  // extern "C"
