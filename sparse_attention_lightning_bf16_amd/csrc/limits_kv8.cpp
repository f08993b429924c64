// Host-side plans of the 8-bit cache kernels: how attention splits its work
// and what workspaces the calls need.  Plain C++, shared by the C ABI's
// validation and the launchers.
#include "launch_kv8.h"

namespace lix {

// Rows to a wave: 32 where their accumulators leave room for two waves per
// SIMD (D <= 128) and there are more than 16, else 16.  Many rows: workgroups
// of 4 waves that share the conversion of their keys (2 where a query's heads
// fill no more).  Where the rows make fewer waves than fill the card (8 for
// each of 256 CUs), the keys are split into parts of at least 128 keys.
AttendPlan attend_plan(int B, int S, int Hq, int Hkv, int D, int page, int max_pages, int topk) {
    constexpr long kWaves = 2048, kPartKeys = 128, kMaxParts = 256;
    const int G = Hq / Hkv;
    const long rows = topk > 0 ? G : (long)S * G;
    const long keys = topk > 0 ? topk : (long)max_pages * page;
    AttendPlan p{};
    p.tiles = rows > 16 && D <= 128 ? 2 : 1;
    if (topk > 0) p.waves = rows <= 16 ? 0 : rows <= 2 * 16 * p.tiles ? 2 : 4;
    else p.waves = rows > 8 * 16 * p.tiles ? 8 : rows > 64 ? 4 : 0;
    const long group = 16L * p.tiles * (p.waves > 0 ? p.waves : 1);
    p.row_tiles = (int)((rows + group - 1) / group);
    p.tasks = (long)B * Hkv * (topk > 0 ? S : 1);
    const long waves = p.tasks * p.row_tiles * (p.waves > 0 ? p.waves : 1);
    long parts = (kWaves + waves - 1) / waves;
    const long most = (keys + kPartKeys - 1) / kPartKeys;
    if (parts > most) parts = most;
    if (parts > kMaxParts) parts = kMaxParts;
    p.parts = (int)parts;
    p.workspace_bytes = parts > 1 ? p.tasks * parts * rows * (D + 2) * 4 : 0;
    return p;
}

EvictLayout evict_layout(int B, int Hkv, int width, int keep, int recent, int sinks) {
    auto up = [](long x) { return (x + 255) & ~255L; };
    const long rows = (long)B * Hkv;
    EvictLayout ly{};
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
