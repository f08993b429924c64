// C ABI of rotary positions (lix_rotary.h): validation and dispatch, on the
// host before any launch as in api.cpp.
#include "launch_kv8.h"
#include "lix_rotary.h"
#include "validate.h"

extern "C" int lix_rotary(const void* x, long long x_s0, long long x_s1, long long x_sh, const int32_t* positions,
               long long p_s0, long long p_s1, const double* inv_freq, int N0, int N1, int H, int D, int rot, int start,
               int layout, float scale, int inverse, int dtype, void* out, long long o_s0, long long o_s1,
               long long o_sh, hipStream_t stream) {
    using namespace lix;
    if (!x || !positions || !inv_freq || !out) return LIX_ERR_NULL;
    if (N0 <= 0 || N1 <= 0 || H <= 0 || D <= 0 || rot < 2 || rot % 2 != 0 || start < 0 || rot > D || start > D - rot)
        return LIX_ERR_SHAPE;
    if ((layout != LIX_ROTARY_HALF && layout != LIX_ROTARY_INTERLEAVED) ||
        (dtype != LIX_BF16 && dtype != LIX_FP16 && dtype != LIX_FP32))
        return LIX_ERR_SHAPE;
    // strides below 2^40 keep every offset inside int64
    const long long lim = 1LL << 40;
    for (long long s : {x_s0, x_s1, x_sh, p_s0, p_s1, o_s0, o_s1, o_sh}) {
        if (s < 0) return LIX_ERR_SHAPE;
        if (s > lim / D) return LIX_ERR_UNSUPPORTED;
    }
    if (D > 1024 || !fits(N0, N1, H, D) || (long long)N0 * N1 > (1LL << 30) || (long long)H * D > (1LL << 24))
        return LIX_ERR_UNSUPPORTED;
    const uintptr_t size = dtype == LIX_FP32 ? 4 : 2;
    if (!aligned(x, size) || !aligned(out, size) || !aligned(positions, 4) || !aligned(inv_freq, 8))
        return LIX_ERR_UNSUPPORTED;
    const int st = check_device({x, positions, inv_freq, out});
    if (st != LIX_OK) return st;
    RotaryArgs a{x, (long)x_s0, (long)x_s1, (long)x_sh, positions, (long)p_s0, (long)p_s1, inv_freq, N0, N1, H, D,
                 rot, start, layout, scale, inverse, dtype, out, (long)o_s0, (long)o_s1, (long)o_sh, stream};
    return launch_status(launch_rotary(a));
}
