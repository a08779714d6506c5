// Device-side building blocks of the attention kernels (gfx950 only).
//
// Every pass is a chain of small matrix products on v_mfma_f32_16x16x4_f32
// (D = A B + C; A 16 x 4, B 4 x 16).  Lane l holds A[l % 16][l / 16], B[l / 16][l
// % 16] and D[4 (l / 16) + j][l % 16], j = 0..3.  A pass keeps 16 of its own
// rows (queries, or keys) as the columns of D and streams the other side
// through the rows of D:
//   - scores: A = streamed rows, contraction over d.  The order of d within
//     the contraction is free as long as A and B agree: lane group h = l / 16
//     takes d = 16 c + 4 h + s in step s, so that a 16-byte read feeds four
//     steps;
//   - results: A = streamed rows transposed, contraction over the streamed
//     rows.  Step j takes row 4 h + j, which is the row of D that the same
//     lane holds, so that a score's registers are B as they are, with no move
//     between lanes.  The rows of this A (the result's d) are numbered so that
//     a read of VT neighbouring floats feeds VT tiles: tile (c, u) has d = 16
//     VT c + VT m + u in row m.
// One row-major copy of the streamed tile in LDS serves both.
#pragma once

#include "emu_attn_launch.h"
#include "emu_block_device.h"

namespace emu {

__device__ __forceinline__ f32x4_t mfma4(float a, float b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

constexpr float kLog2e = 1.44269502162933349609375f;
__device__ __forceinline__ float minus_inf() { return -__builtin_inff(); }

// e^x, x <= 0.  The product's rounding costs |x| 2^-24 of the value, e^x |x|
// 2^-24 < 2^-25 of the row's largest: below the rounding of the sums it enters.
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

// ND tiles of 16 cover a head (dim <= 16 ND); LD is the tile's row length in
// LDS: four more than a multiple of 16, so that the 16 rows of a score's reads
// lie on different banks.
template <int ND>
struct Head {
    static constexpr int VT = ND % 4 == 0 ? 4 : ND % 2 == 0 ? 2 : 1;
    static constexpr int NC = ND / VT;
    static constexpr int LD = 16 * ND + 4;
};

// A wave's own row as the B operand of scores.
template <int ND>
__device__ __forceinline__ void load_own(f32x4_t (&f)[ND], const float* row, bool valid, int h, int dim)
{
#pragma unroll
    for (int c = 0; c < ND; ++c) f[c] = valid ? load4(row, 16 * c + 4 * h, dim) : f32x4_t{};
}

// acc[n] += (16 streamed rows at `tile`) . own[n]
template <int ND, int NT>
__device__ __forceinline__ void scores(const float* tile, int m, int h, const f32x4_t (&own)[NT][ND], f32x4_t (&acc)[NT])
{
    const float* at = tile + m * Head<ND>::LD + 4 * h;
#pragma unroll
    for (int c = 0; c < ND; ++c) {
        const f32x4_t a = *reinterpret_cast<const f32x4_t*>(at + 16 * c);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n] = mfma4(a[s], own[n][c][s], acc[n]);
    }
}

// acc[n] += (16 streamed rows at `tile`)^T . w[n], w as scores() leaves it
template <int ND, int NT>
__device__ __forceinline__ void results(const float* tile, int m, int h, const f32x4_t (&w)[NT], f32x4_t (&acc)[NT][ND])
{
    constexpr int VT = Head<ND>::VT;
    typedef float vec_t __attribute__((ext_vector_type(VT)));
    const float* at = tile + 4 * h * Head<ND>::LD + VT * m;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < Head<ND>::NC; ++c) {
            float a[VT];
            if constexpr (VT == 1) {
                a[0] = at[j * Head<ND>::LD + 16 * c];
            } else {
                const vec_t v = *reinterpret_cast<const vec_t*>(at + j * Head<ND>::LD + 16 * VT * c);
#pragma unroll
                for (int u = 0; u < VT; ++u) a[u] = v[u];
            }
#pragma unroll
            for (int u = 0; u < VT; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][c * VT + u] = mfma4(a[u], w[n][j], acc[n][c * VT + u]);
        }
}

// A result's column (results()) to a row of `dim` floats, times f.
template <int ND>
__device__ __forceinline__ void store_own(const f32x4_t (&acc)[ND], float f, float* row, int h, int dim)
{
    constexpr int VT = Head<ND>::VT;
#pragma unroll
    for (int c = 0; c < Head<ND>::NC; ++c) {
        float v[4 * VT];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < VT; ++u) v[j * VT + u] = acc[c * VT + u][j] * f;
#pragma unroll
        for (int e = 0; e < VT; ++e)
            store4(row, 16 * VT * c + 4 * VT * h + 4 * e, dim, f32x4_t{v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]});
    }
}

template <int ND, int NT>
__device__ __forceinline__ void clear(f32x4_t (&acc)[NT][ND])
{
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < ND; ++t) acc[n][t] = f32x4_t{};
}

// ---- teams --------------------------------------------------------------------------
//
// A workgroup of 256 threads is four teams of one wave, each with a share of
// LDS and a piece of work of its own, or one team of four waves.

template <int W>
struct Team {
    static constexpr int kThreads = 64 * W, kTeams = 4 / W;
    static __device__ __forceinline__ int index() { return W == 4 ? 0 : (int)(threadIdx.x >> 6); }
    static __device__ __forceinline__ int thread() { return (int)(threadIdx.x & (kThreads - 1)); }
    static __device__ __forceinline__ int wave() { return W == 4 ? (int)(threadIdx.x >> 6) : 0; }
    // LDS written by the team is seen by the team.  (LDS accesses of one wave
    // complete in order: one wave only has to keep the compiler from moving
    // them.)
    static __device__ __forceinline__ void sync()
    {
        if constexpr (W == 4) {
            __syncthreads();
        } else {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
    }
};

// f(piece) for the team's pieces of 0 .. n-1.  Workgroup b runs on XCD b % 8,
// each with an L2 of its own: neighbouring pieces, which read the same other
// side, go to one XCD.
template <int W, class F>
__device__ __forceinline__ void each_piece(int64_t n, F&& f)
{
    const int64_t groups = (n + Team<W>::kTeams - 1) / Team<W>::kTeams, per = (groups + 7) / 8;
    for (int64_t b = blockIdx.x; b < 8 * per; b += gridDim.x) {
        const int64_t group = (b & 7) * per + (b >> 3), piece = group * Team<W>::kTeams + Team<W>::index();
        if (group < groups && piece < n) f(piece);
    }
}

// Workgroups for n pieces: all of them at once, up to what a launch holds.
template <int W>
inline unsigned attn_grid(int64_t n)
{
    const int64_t groups = (n + Team<W>::kTeams - 1) / Team<W>::kTeams, all = (groups + 7) / 8 * 8;
    return (unsigned)(all < ((int64_t)1 << 22) ? all : (int64_t)1 << 22);
}

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
    const int q = (int)((unsigned)r / (unsigned)a.share);
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

// Rows of a streamed tile: fewer where four teams of one wave share the LDS.
template <int ND, int W>
struct StreamTile {
    static constexpr int kRows = W == 1 && ND >= 4 ? 16 : 32;
};

// A streamed tile of ROWS rows on its way to LDS: fetch() requests it into
// registers, put() writes it.  where(row) is the row's address, null for a
// row of zeros.
template <int ND, int ROWS, int THREADS>
struct Tile {
    static constexpr int kQuads = 4 * ND, kAll = ROWS * kQuads, kEach = (kAll + THREADS - 1) / THREADS;
    // (half of a team of four waves has a piece of the narrowest tiles)
    static constexpr bool kSome = kAll % THREADS != 0;
    f32x4_t v[kEach];

    template <class F>
    __device__ __forceinline__ void fetch(int thread, int dim, F&& where)
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = thread + i * THREADS, row = at / kQuads, col = at % kQuads * 4;
            const float* p = kSome && at >= kAll ? nullptr : where(row);
            v[i] = p != nullptr ? load4(p, col, dim) : f32x4_t{};
        }
    }
    __device__ __forceinline__ void put(int thread, float* tile) const
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = thread + i * THREADS, row = at / kQuads, col = at % kQuads * 4;
            if (!kSome || at < kAll) *reinterpret_cast<f32x4_t*>(tile + row * Head<ND>::LD + col) = v[i];
        }
    }
};

// f.template operator()<ND, W, NT>() for a head and plan; WIDE: tiles of 16
// per wave that the registers hold of the widest heads, as the plan
// has it.
template <int WIDE, class F>
inline void with_shape(int dim, const AttnPlan& p, F&& f)
{
    const auto tiles = [&]<int ND>() {
        if constexpr (ND < 8 || WIDE == 2) {
            if (p.tiles == 2 && p.waves == 1) return f.template operator()<ND, 1, 2>();
            if (p.tiles == 2) return f.template operator()<ND, 4, 2>();
        }
        if (p.waves == 1) return f.template operator()<ND, 1, 1>();
        return f.template operator()<ND, 4, 1>();
    };
    if (dim <= 16)
        tiles.template operator()<1>();
    else if (dim <= 32)
        tiles.template operator()<2>();
    else if (dim <= 64)
        tiles.template operator()<4>();
    else
        tiles.template operator()<8>();
}

}  // namespace emu
