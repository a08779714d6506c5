// Rotary positions (include/emu_attention.h).
//
// Bound by memory: an element is read and written once.  The angle is the
// product of the position and the frequency, a 64-bit fraction of a turn,
// modulo 2^64: what is left of it is exact at any position, where an FP32
// angle of a million radians has lost all of its fraction.  A thread makes the
// cosine and sine of its pairs once and takes them through the heads of its
// token.
#include "emu_attn_launch.h"
#include "emu_block_device.h"

namespace emu {
namespace {

struct Turn {
    float cos, sin;
};

// The cosine and sine of `turn` 2^-64 turns, times f.
__device__ __forceinline__ Turn turn_of(uint64_t turn, float f, bool inverse)
{
    // the nearest quarter turn, and what is left: an eighth at most, so that
    // its upper 32 bits lose 2^-28 turns in FP32
    const uint64_t quarter = (turn + ((uint64_t)1 << 61)) >> 62;
    const float rest = (float)(int32_t)((turn - (quarter << 62)) >> 32) * 0x1p-31f;   // (half turns)
    float s, c;
    sincospif(rest, &s, &c);
    const float cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
    const float cos = quarter == 1 || quarter == 2 ? -cs : cs, sin = (quarter >= 2) != inverse ? -sn : sn;
    return {cos * f, sin * f};
}

// Work items of a token and head: groups of four elements, rotated ones first.
// HALF: group i is elements 4 i .. and pairs + 4 i ..; INTERLEAVED: pairs 2 i,
// 2 i + 1; then the rest of the head in groups of four.
template <int LAYOUT>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, int groups, int copies, int heads_each, int head_parts)
{
    const int64_t n = a.batch * a.tokens * head_parts * (groups + copies);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t at = i / (groups + copies);
        const int group = (int)(i - at * (groups + copies));
        const int64_t token_at = at / head_parts;
        const int h0 = (int)(at - token_at * head_parts) * heads_each;
        const int64_t b = token_at / a.tokens, t = token_at - b * a.tokens;
        const int h1 = h0 + heads_each < a.heads ? h0 + heads_each : a.heads;
        const float* x = a.x.data + (b * a.x.batch + t * a.x.token);
        float* y = a.y + (b * a.tokens + t) * a.heads * a.dim;
        if (group >= groups) {
            const int col = 2 * a.pairs + 4 * (group - groups);
            for (int h = h0; h < h1; ++h) store4(y + (int64_t)h * a.dim, col, a.dim, load4(x + h * a.x.head, col, a.dim));
            continue;
        }
        const uint64_t pos = (uint64_t)a.positions[b * a.pos_b + t * a.pos_t];
        constexpr int N = LAYOUT == EMU_ROTARY_HALF ? 4 : 2;
        Turn turn[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int pair = N * group + e;
            turn[e] = turn_of(pair < a.pairs ? pos * a.turns[pair] : 0, a.magnitude, a.inverse != 0);
        }
        for (int h = h0; h < h1; ++h) {
            const float* xr = x + h * a.x.head;
            float* yr = y + (int64_t)h * a.dim;
            if constexpr (LAYOUT == EMU_ROTARY_HALF) {
                const f32x4_t p = load4(xr, 4 * group, a.pairs), q = load4(xr + a.pairs, 4 * group, a.pairs);
                f32x4_t u, v;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    u[e] = __builtin_fmaf(p[e], turn[e].cos, -(q[e] * turn[e].sin));
                    v[e] = __builtin_fmaf(p[e], turn[e].sin, q[e] * turn[e].cos);
                }
                store4(yr, 4 * group, a.pairs, u);
                store4(yr + a.pairs, 4 * group, a.pairs, v);
            } else {
                const f32x4_t p = load4(xr, 4 * group, 2 * a.pairs);
                f32x4_t u;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    u[2 * e] = __builtin_fmaf(p[2 * e], turn[e].cos, -(p[2 * e + 1] * turn[e].sin));
                    u[2 * e + 1] = __builtin_fmaf(p[2 * e], turn[e].sin, p[2 * e + 1] * turn[e].cos);
                }
                store4(yr, 4 * group, 2 * a.pairs, u);
            }
        }
    }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t s)
{
    const int groups = a.layout == EMU_ROTARY_HALF ? (a.pairs + 3) / 4 : (a.pairs + 1) / 2;
    const int copies = (a.dim - 2 * a.pairs + 3) / 4;
    // heads that share a thread's cosines, fewer where threads are few
    int each = a.heads;
    while (each > 1 && a.batch * a.tokens * ((a.heads + each - 1) / each) * (groups + copies) < 256 * 1024) each = (each + 1) / 2;
    const int parts = (a.heads + each - 1) / each;
    const int64_t wgs = (a.batch * a.tokens * parts * (groups + copies) + 255) / 256;
    const unsigned grid = (unsigned)(wgs < 65536 ? wgs : 65536);
    if (a.layout == EMU_ROTARY_HALF)
        rotary_kernel<EMU_ROTARY_HALF><<<grid, 256, 0, s>>>(a, groups, copies, each, parts);
    else
        rotary_kernel<EMU_ROTARY_INTERLEAVED><<<grid, 256, 0, s>>>(a, groups, copies, each, parts);
    return hipGetLastError();
}

}  // namespace emu
