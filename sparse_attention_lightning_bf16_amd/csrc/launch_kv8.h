// Internal launch interface between the C ABI (api_rotary.cpp, api_kv8.cpp)
// and the kernels of rotary positions and of the 8-bit cache.  Arguments have
// been validated by the caller; launchers only enqueue.  Plain C++.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "lix_rotary.h"

namespace lix {

struct RotaryArgs {
    const void* x;
    long x_s0, x_s1, x_sh;
    const int32_t* positions;
    long p_s0, p_s1;
    const double* inv_freq;
    int N0, N1, H, D, rot, start, layout;
    float scale;
    int inverse, dtype;
    void* out;
    long o_s0, o_s1, o_sh;
    hipStream_t stream;
};
hipError_t launch_rotary(const RotaryArgs& p);

// The cache as a kernel sees it.
struct KV8Pages {
    uint8_t* k;               // e4m3 [num_pages, Hkv, page, D]
    uint8_t* v;
    float* k_scale;           // fp32 [num_pages, Hkv]
    float* v_scale;
    int num_pages, page_shift;   // page = 1 << page_shift tokens
    int Hkv, D;
    const int32_t* table;     // [B, max_pages]
    int max_pages;
    const int32_t* lens;      // [B]
};

struct AppendArgs {
    const void* x[2];         // k, v
    long sb[2], ss[2], sh[2];
    int dtype, B, S;
    KV8Pages c;
    const int32_t* new_lens;  // [B] or null
    hipStream_t stream;
};
hipError_t launch_kv8_append(const AppendArgs& p);

struct QueryArgs {
    const void* q;
    long sb, ss, sh;
    int dtype, B, S, Hq, G;   // G = Hq / Hkv
    const int32_t* q_start;   // [B] or null
    const int32_t* q_lens;    // [B] or null
    int ratio;
    float scale_log2;         // scale * log2(e)
};

struct AttendArgs {
    QueryArgs q;
    KV8Pages c;
    const int32_t* indices;   // [B, S, topk] or null
    int topk;
    void* out;
    float* lse;
    float* workspace;
    hipStream_t stream;
};
constexpr int kMaxParts = 256;
// How lix_kv8_attention splits its work.
struct AttendPlan {
    int waves;                // of a workgroup that shares its keys through LDS; 0: that shares its rows
    int tiles;                // 16-row tiles of a wave
    int row_tiles;            // workgroups for the rows of one (sequence, key head) or query
    int parts;                // parts of the keys, at most kMaxParts
    long tasks;               // (sequence, key head[, query]) groups
    long workspace_bytes;
};
AttendPlan attend_plan(int B, int S, int Hq, int Hkv, int D, int page, int max_pages, int topk);
hipError_t launch_kv8_attention(const AttendArgs& p, const AttendPlan& plan);
// The part of launch_kv8_attention for plans with waves > 0, before any joining.
hipError_t launch_kv8_tiles(const AttendArgs& p, const AttendPlan& plan);

struct WeighArgs {
    QueryArgs q;
    KV8Pages c;
    const float* lse;
    float* weights;
    int width, accumulate;
    long cap;                 // tokens of a table row
    int parts;                // of the rows (WeighPlan)
    float* workspace;         // [parts, B, Hkv, cap], parts > 1
    hipStream_t stream;
};
// How lix_kv8_token_weights splits its work: parts of the rows, or, for one
// tile of 16 rows, the keys of a wave (range > 0).
struct WeighPlan {
    int parts, range;
    long workspace_bytes;
};
WeighPlan weigh_plan(int B, int S, int Hq, int Hkv, int D, int page, int max_pages);
hipError_t launch_kv8_token_weights(const WeighArgs& p, const WeighPlan& plan);

struct EvictArgs {
    KV8Pages c;
    int B;
    const float* weights;
    int width;
    const int32_t* new_table;
    int new_max_pages;
    int keep, recent, sinks;
    int32_t* new_lens;
    int32_t* kept;
    float* new_weights;
    void* workspace;
    hipStream_t stream;
};
// lix_kv8_evict: whether its rows are selected by the row top-k, the byte
// offsets of the parts of the workspace that this takes, and the tokens it
// selects of a row (middle).
struct EvictLayout {
    bool by_topk;
    long begin, end, scores, indices, total;
    int middle;
};
EvictLayout evict_layout(int B, int Hkv, long cap, int width, int keep, int recent, int sinks);
hipError_t launch_kv8_evict(const EvictArgs& p, const EvictLayout& layout);

}  // namespace lix
