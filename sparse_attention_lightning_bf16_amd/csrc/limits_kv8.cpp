// Host-side plans of the 8-bit cache kernels: how attention splits its work
// and what workspaces the calls need.  Plain C++, shared by the C ABI's
// validation and the launchers.
#include "launch_kv8.h"

namespace lix {

// Rows to a wave: 32 where their accumulators leave room for two waves per
// SIMD (D <= 128) and there are more than 16, else 16.  Many rows: workgroups
// of 8 or 4 waves that share the conversion of their keys, each wave with its
// own rows (16 heads of a query over its list).  Few: workgroups of 4 waves
// that share the rows and take turns at the keys.
//
// Where the rows make too few workgroups, the keys are split into parts of at
// least 1024 keys: for many rows until the card is full (2048 waves), for few
// until there are 1024 workgroups, two for each place on the card.
AttendPlan attend_plan(int B, int S, int Hq, int Hkv, int D, int page, int max_pages, int topk) {
    constexpr long kWaves = 2048, kGroups = 1024, kPartKeys = 1024;
    const int G = Hq / Hkv;
    const long rows = topk > 0 ? G : (long)S * G;
    const long keys = topk > 0 ? topk : (long)max_pages * page;
    AttendPlan p{};
    p.tiles = rows > 16 && D <= 128 ? 2 : 1;
    if (topk > 0) {
        p.tiles = 1;
        p.waves = rows > 16 ? 4 : 0;
    } else {
        p.waves = rows > 8 * 16 * p.tiles ? 8 : rows > 64 ? 4 : 0;
    }
    const long group = 16L * p.tiles * (p.waves > 0 ? p.waves : 1);
    p.row_tiles = (int)((rows + group - 1) / group);
    p.tasks = (long)B * Hkv * (topk > 0 ? S : 1);
    const long groups = p.tasks * p.row_tiles;
    const long wanted = p.waves > 0 ? kWaves / p.waves : kGroups;
    long parts = (wanted + groups - 1) / groups;
    const long most = keys < kPartKeys ? 1 : keys / kPartKeys;
    if (parts > most) parts = most;
    if (parts > kMaxParts) parts = kMaxParts;
    p.parts = (int)parts;
    p.workspace_bytes = parts > 1 ? p.tasks * parts * rows * (D + 2) * 4 : 0;
    return p;
}

// One tile of rows: ranges of 1024 keys to a wave (64 lookups of 16), shorter
// ones down to 64 where that leaves fewer than 8192 waves.  More rows: 256 keys
// (128 for D = 256) to a workgroup, the rows in parts until there are 2048
// workgroups, at least eight tiles of 16 rows to a part.
WeighPlan weigh_plan(int B, int S, int Hq, int Hkv, int D, int page, int max_pages) {
    const long cap = (long)max_pages * page, pairs = (long)B * Hkv, rows = (long)S * (Hq / Hkv);
    WeighPlan p{};
    p.parts = 1;
    if (rows <= 16) {
        p.range = 1024;
        while (p.range > 64 && pairs * ((cap + p.range - 1) / p.range) < 8192) p.range /= 2;
        return p;
    }
    const long keys = D <= 128 ? 256 : 128;
    const long groups = pairs * ((cap + keys - 1) / keys);
    long parts = (2048 + groups - 1) / groups;
    const long most = (rows + 127) / 128;
    if (parts > most) parts = most;
    p.parts = (int)parts;
    p.workspace_bytes = parts > 1 ? parts * pairs * cap * 4 : 0;
    return p;
}

EvictLayout evict_layout(int B, int Hkv, long cap, int width, int keep, int recent, int sinks) {
    auto up = [](long x) { return (x + 255) & ~255L; };
    const long rows = (long)B * Hkv;
    EvictLayout ly{};
    ly.by_topk = cap > 32768;
    if (!ly.by_topk) return ly;
    // a row with more than keep tokens has more than keep - recent - sinks in the
    // middle, and width covers them all
    const int middle = keep - recent - sinks;
    ly.middle = middle < width ? middle : width;
    ly.begin = 0;
    ly.end = ly.begin + up(rows * 4);
    ly.scores = ly.end + up(rows * 4);
    ly.indices = ly.scores + up(rows * ly.middle * 4);
    ly.total = ly.indices + up(rows * ly.middle * 4);
    return ly;
}

}  // namespace lix
