// Rotary positions (include/emu_attention.h).
//
// Bound by memory: an element is read and written once; 552,960 tokens of 8 x 32
// in 242 us (4.7 TB/s), 4 x 16,381 of 16 x 128 in 199 (5.4).  The angle is the
// product of the position and the frequency, a 64-bit fraction of a turn,
// modulo 2^64: what is left of it is exact at any position, where an FP32
// angle of a million radians has lost all of its fraction.
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

constexpr int kTokens = 32;   // most tokens of a workgroup
constexpr int kTurns = 1024;  // and cosines of them

// A workgroup's tokens: first their cosines and sines, shared by all heads,
// then the heads in groups of four elements (HALF: elements 4 i .. and pairs +
// 4 i ..; INTERLEAVED: pairs 2 i, 2 i + 1; then what is copied), as they follow
// each other in memory, kAtOnce groups of a thread requested together.
// blockIdx.y: which of the chunks of `chunk` groups, of heads too wide to
// share their cosines at once.
template <int LAYOUT>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, int tokens_each, int groups, int copies, int chunk)
{
    constexpr int N = LAYOUT == EMU_ROTARY_HALF ? 4 : 2, kAtOnce = 4;   // pairs of a group
    __shared__ Turn turns[kTurns];
    __shared__ int64_t from[kTokens];
    const int64_t all = a.batch * a.tokens;
    const int g0 = blockIdx.y * chunk, rest = groups + copies - g0, here = rest < chunk ? rest : chunk;
    const int turned = g0 >= groups ? 0 : groups - g0 < here ? groups - g0 : here;
    for (int64_t first = (int64_t)blockIdx.x * tokens_each; first < all; first += (int64_t)gridDim.x * tokens_each) {
        const int count = (int)(all - first < tokens_each ? all - first : tokens_each);
        __syncthreads();   // the previous tokens' have been read
        for (int i = threadIdx.x; i < count * N * turned; i += 256) {
            const int token = (int)((unsigned)i / (unsigned)(N * turned)), pair = i - token * N * turned + N * g0;
            const int64_t b = (first + token) / a.tokens, t = first + token - b * a.tokens;
            const uint64_t pos = pair < a.pairs ? (uint64_t)a.positions[b * a.pos_b + t * a.pos_t] : 0;
            turns[i] = turn_of(pair < a.pairs ? pos * a.turns[pair] : 0, a.magnitude, a.inverse != 0);
        }
        if ((int)threadIdx.x < count) {
            const int64_t b = (first + threadIdx.x) / a.tokens, t = first + threadIdx.x - b * a.tokens;
            from[threadIdx.x] = b * a.x.batch + t * a.x.token;
        }
        __syncthreads();
        const int per_token = a.heads * here, n = count * per_token;
        for (int i0 = threadIdx.x; i0 < n; i0 += 256 * kAtOnce) {
            f32x4_t p[kAtOnce], q[kAtOnce];
            int token[kAtOnce], group[kAtOnce];
            float* y[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int i = i0 + 256 * k < n ? i0 + 256 * k : i0;
                token[k] = (int)((unsigned)i / (unsigned)per_token);
                const int in = i - token[k] * per_token, head = (int)((unsigned)in / (unsigned)here);
                group[k] = in - head * here;
                const float* const x = a.x.data + (from[token[k]] + head * a.x.head);
                y[k] = a.y + ((first + token[k]) * a.heads + head) * a.dim;
                const int g = g0 + group[k];
                if (group[k] >= turned) {
                    p[k] = load4(x, 2 * a.pairs + 4 * (g - groups), a.dim);
                } else if constexpr (LAYOUT == EMU_ROTARY_HALF) {
                    p[k] = load4(x, 4 * g, a.pairs);
                    q[k] = load4(x + a.pairs, 4 * g, a.pairs);
                } else {
                    p[k] = load4(x, 4 * g, 2 * a.pairs);
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (i0 + 256 * k >= n) continue;
                const int g = g0 + group[k];
                const Turn* const turn = turns + (token[k] * turned + group[k]) * N;
                if (group[k] >= turned) {
                    store4(y[k], 2 * a.pairs + 4 * (g - groups), a.dim, p[k]);
                } else if constexpr (LAYOUT == EMU_ROTARY_HALF) {
                    f32x4_t u, v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        u[e] = __builtin_fmaf(p[k][e], turn[e].cos, -(q[k][e] * turn[e].sin));
                        v[e] = __builtin_fmaf(p[k][e], turn[e].sin, q[k][e] * turn[e].cos);
                    }
                    store4(y[k], 4 * g, a.pairs, u);
                    store4(y[k] + a.pairs, 4 * g, a.pairs, v);
                } else {
                    f32x4_t u;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        u[2 * e] = __builtin_fmaf(p[k][2 * e], turn[e].cos, -(p[k][2 * e + 1] * turn[e].sin));
                        u[2 * e + 1] = __builtin_fmaf(p[k][2 * e], turn[e].sin, p[k][2 * e + 1] * turn[e].cos);
                    }
                    store4(y[k], 4 * g, 2 * a.pairs, u);
                }
            }
        }
    }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t s)
{
    const int pairs = a.layout == EMU_ROTARY_HALF ? 4 : 2;   // of a group
    const int groups = (a.pairs + pairs - 1) / pairs;
    const int copies = (int)(((int64_t)a.dim - 2 * a.pairs + 3) / 4);
    // groups at once, and tokens: 16 KB of elements (or what is there for 1,024
    // workgroups), as far as their cosines fit
    const int chunk = groups + copies < kTurns / 4 ? groups + copies : kTurns / 4;
    const int64_t all = a.batch * a.tokens, work = (int64_t)a.heads * chunk;
    int64_t each = 1024 / work;
    if (each > (all + 1023) / 1024) each = (all + 1023) / 1024;
    if (each > kTokens) each = kTokens;
    if (each * chunk * pairs > kTurns) each = kTurns / (chunk * pairs);
    if (each < 1) each = 1;
    const int64_t wgs = (all + each - 1) / each;
    const dim3 grid((unsigned)(wgs < ((int64_t)1 << 20) ? wgs : (int64_t)1 << 20), (unsigned)((groups + copies + chunk - 1) / chunk));
    if (a.layout == EMU_ROTARY_HALF)
        rotary_kernel<EMU_ROTARY_HALF><<<grid, 256, 0, s>>>(a, (int)each, groups, copies, chunk);
    else
        rotary_kernel<EMU_ROTARY_INTERLEAVED><<<grid, 256, 0, s>>>(a, (int)each, groups, copies, chunk);
    return hipGetLastError();
}

}  // namespace emu
