// What the attention kernels share on the device (gfx950 only).
//
// Every pass is a chain of small matrix products D = A B + C whose 16 x 16
// result has D[4 (l / 16) + j][l % 16], j = 0..3, in lane l. A pass keeps 16 of
// its own rows (queries, or keys) as the columns of D and streams the other
// side through the rows of D, so that a softmax's maxima, sums and factors are
// per lane, and a score's registers are the next product's B as they are: its
// contraction over the streamed rows may take them in any order, so lane group
// l / 16 takes those that it holds.
#pragma once

#include "emu_attn_launch.h"
#include "emu_block_device.h"

namespace emu {

constexpr float kLog2e = 1.44269502162933349609375f;
__device__ __forceinline__ float minus_inf() { return -__builtin_inff(); }

// e^x of a score less its row's maximum, which may lag by up to 1 (kSlack of the
// forward pass, whose maximum the other passes take over).  The product's
// rounding, and log2(e)'s own, cost up to 1.22 |x| 2^-24 of the value: for x <= 0
// less than 2^-25 of the row's largest weight, below the rounding of the sums it
// enters, and for x up to 1 less than 2^-24 of the weight itself.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

__device__ __forceinline__ float max_lane16(float x)
{
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float max_lane32(float x)
{
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
// Over the four lane groups, which hold the rows of a column of D.
__device__ __forceinline__ float column_max(float x) { return max_lane32(max_lane16(x)); }
__device__ __forceinline__ float column_sum(float x) { return add_lane32(add_lane16(x)); }

// ---- teams --------------------------------------------------------------------------
//
// A team of W waves has pieces of work of its own; a workgroup is one team, or
// several of one wave, each with a share of LDS.

template <int W, int TEAMS = 1>
struct Team {
    static_assert(W == 1 || TEAMS == 1, "teams of more waves have a workgroup of their own");
    static constexpr int kThreads = 64 * W, kTeams = TEAMS, kGroup = kThreads * TEAMS;
    static __device__ __forceinline__ int index() { return TEAMS == 1 ? 0 : (int)(threadIdx.x >> 6); }
    static __device__ __forceinline__ int thread() { return (int)(threadIdx.x & (kThreads - 1)); }
    static __device__ __forceinline__ int wave() { return W == 1 ? 0 : (int)(threadIdx.x >> 6); }
    // LDS written by the team is seen by the team.  (LDS accesses of one wave
    // complete in order: one wave only has to keep the compiler from moving
    // them.)
    static __device__ __forceinline__ void sync()
    {
        if constexpr (W > 1) {
            __syncthreads();
        } else {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
    }

    // f(piece) for the team's pieces of 0 .. n-1. Workgroup b runs on XCD b %
    // 8, each with an L2 of its own: the pieces of a run, which read the same
    // other side, go to one XCD, and the runs are dealt to the XCDs in turn, so
    // that sequences of different lengths lie on all of them (21 x 8 heads of 200
    // x up to 1,918 x 48, second order: 601 us by rows and 401 by keys with an
    // eighth of the pieces for each XCD, 451 and 307 so).
    template <class F>
    static __device__ __forceinline__ void each_piece(int64_t n, int64_t run, F&& f)
    {
        const int64_t groups = (n + TEAMS - 1) / TEAMS, all = (groups + 8 * run - 1) / (8 * run) * (8 * run);
        for (int64_t b = blockIdx.x; b < all; b += gridDim.x) {
            const int64_t i = b >> 3, turn = i < ((int64_t)1 << 31) && run < ((int64_t)1 << 31) ? (unsigned)i / (unsigned)run : i / run;
            const int64_t group = (turn * 8 + (b & 7)) * run + (i - turn * run), piece = group * TEAMS + index();
            if (group < groups && piece < n) f(piece);
        }
    }

    // Workgroups for n pieces: all of them at once, up to what a launch holds.
    static unsigned grid(int64_t n, int64_t run)
    {
        const int64_t groups = (n + TEAMS - 1) / TEAMS, all = (groups + 8 * run - 1) / (8 * run) * (8 * run);
        return (unsigned)(all < ((int64_t)1 << 21) ? all : (int64_t)1 << 21);
    }
};

// Keys that may take part of sequence b.
__device__ __forceinline__ int keys_of(const AttnArgs& a, int b)
{
    if (a.lengths == nullptr) return a.keys;
    const int64_t n = a.lengths_64 ? static_cast<const int64_t*>(a.lengths)[b] : static_cast<const int32_t*>(a.lengths)[b];
    return n < 0 ? 0 : n > a.keys ? a.keys : (int)n;
}

// What key j adds to a score: its bias, -infinity if it takes no part.
__device__ __forceinline__ float key_term(const AttnArgs& a, int b, int j, int limit)
{
    if (j >= limit) return minus_inf();
    if (a.mask != nullptr && a.mask[b * a.mask_b + j * a.mask_k] == 0) return minus_inf();
    return a.bias != nullptr ? a.bias[b * a.bias_b + j * a.bias_k] : 0.0f;
}

// The team's piece: sequence, key head, piece of its own side, range of the
// other side.
struct Piece {
    int b, g, split;
    int64_t own;
};
__host__ __device__ __forceinline__ int64_t pieces_of(const AttnArgs& a, const AttnPlan& p)
{
    return (int64_t)a.batch * a.kv_heads * p.own * p.splits;
}
__device__ __forceinline__ Piece piece_of(const AttnArgs& a, const AttnPlan& p, int64_t n)
{
    Piece r;
    // (32-bit divisions where they do, as they do for all but enormous calls)
    if (n < ((int64_t)1 << 31) && p.own < ((int64_t)1 << 31)) {
        unsigned i = (unsigned)n;
        r.split = (int)(i % (unsigned)p.splits);
        i /= (unsigned)p.splits;
        r.own = i % (unsigned)p.own;
        i /= (unsigned)p.own;
        r.g = (int)(i % (unsigned)a.kv_heads);
        r.b = (int)(i / (unsigned)a.kv_heads);
    } else {
        r.split = (int)(n % p.splits);
        n /= p.splits;
        r.own = n % p.own;
        n /= p.own;
        r.g = (int)(n % a.kv_heads);
        r.b = (int)(n / a.kv_heads);
    }
    return r;
}

// Range `split` of 0 .. n-1, in whole tiles of `tile`.
__device__ __forceinline__ void range_of(int64_t n, int tile, int splits, int split, int64_t& lo, int64_t& hi)
{
    const int64_t tiles = (n + tile - 1) / tile, per = (tiles + splits - 1) / splits;
    lo = per * split * tile;
    hi = lo + per * tile;
    if (lo > n) lo = n;
    if (hi > n) hi = n;
}

// Row r of a key head: its query and head.
struct RowAt {
    int query, head;
};
__device__ __forceinline__ RowAt row_at(const AttnArgs& a, int g, int64_t r)
{
    if (a.share == 1) return {(int)r, g};
    const int q = a.share_inverse != 0 ? (int)__umulhi((unsigned)r, a.share_inverse) : (int)((unsigned)r / (unsigned)a.share);
    return {q, g * a.share + (int)(r - (int64_t)q * a.share)};
}
__device__ __forceinline__ const float* row_ptr(const emu_heads_t& t, int b, RowAt at)
{
    return t.data + (b * t.batch + at.query * t.token + at.head * t.head);
}
// Its number among the dense rows [batch][queries][heads].
__device__ __forceinline__ int64_t row_index(const AttnArgs& a, int b, RowAt at)
{
    return ((int64_t)b * a.queries + at.query) * a.heads + at.head;
}
__device__ __forceinline__ const float* key_ptr(const emu_heads_t& t, int b, int g, int64_t j)
{
    return t.data + (b * t.batch + j * t.token + g * t.head);
}
__device__ __forceinline__ int64_t key_index(const AttnArgs& a, int b, int g, int64_t j)
{
    return ((int64_t)b * a.keys + j) * a.kv_heads + g;
}

// Partial results of a split: rows' results, then their maxima and sums.
struct ForwardPartial {
    float* o;    // [splits][rows of the call][dim]
    float* ml;   // [splits][rows of the call][2]
};
__host__ __device__ __forceinline__ ForwardPartial forward_partial(const AttnArgs& a, const AttnPlan& p, float* at)
{
    const int64_t n = (int64_t)a.batch * a.queries * a.heads;
    return {at + 2 * p.splits * n, at};
}

}  // namespace emu
