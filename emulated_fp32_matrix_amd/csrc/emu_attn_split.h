// Products of the attention kernels on split operands (gfx950 only).
//
// Each FP32 value is split into three BF16 pieces, hi = R(x), mid = R(x - hi),
// lo = x - hi - mid (R: round to nearest even; exact for |x| from 2^-110, below
// which the lowest pieces run out of BF16's subnormals), and a product is the
// six products of pieces down to 2^-16 of it, accumulated in FP32 by
// v_mfma_f32_16x16x32_bf16. Just above a power of two mid comes near 2^-8 of x
// and lo near 2^-17, so that what is left out, mid lo of either factor and lo lo,
// is up to 1.99 2^-25 of |a b| (over all mantissas), below 2^-24: as much as FP32's
// own rounding of the product. A value beyond BF16's largest finite number has
// hi = that number; infinities give NaN.
//
// Why not the FP32 matrix instruction: it has 1/16 of the rate, 6/16 of it per
// product, and it keeps its SIMD's vector unit from other waves' work
// (measured on 4,096 keys by 2,048 rows of 64: matrix busy + vector active =
// 0.96 with two waves a SIMD), where the softmax and the splits of one wave
// run beside the BF16 products of another.
//
// Layouts: lane l has A[l % 16][8 (l / 16) + i] and B[8 (l / 16) + i][l % 16], i
// = 0..7. Scores: i is d within the step. Results: i < 4 is streamed row 4 (l /
// 16) + i of the first 16, i >= 4 row 4 (l / 16) + i - 4 of the second, which
// a score's registers hold; A comes from the same row-major tile by the LDS's
// transposing read.
#pragma once

#include "emu_attn_device.h"
#include "emu_tile.h"

namespace emu {

typedef short i16x4_t __attribute__((ext_vector_type(4)));

// Four (eight) values' pieces.
struct Split4 {
    u32x2_t p[3];
};
struct Split8 {
    bf16x8_t p[3];
};

// LIMIT: values may pass BF16's largest.
template <bool LIMIT>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo)
{
    hi = LIMIT ? pack_bf16x2(clamp_sat(x0), clamp_sat(x1)) : pack_bf16x2(x0, x1);
    const float r0 = x0 - __uint_as_float(hi << 16), r1 = x1 - __uint_as_float(hi & 0xffff0000u);
    mid = pack_bf16x2(r0, r1);
    lo = pack_bf16x2(r0 - __uint_as_float(mid << 16), r1 - __uint_as_float(mid & 0xffff0000u));
}

__device__ __forceinline__ Split4 split4(f32x4_t v)
{
    uint32_t a[3], b[3];
    split2<true>(v[0], v[1], a[0], a[1], a[2]);
    split2<true>(v[2], v[3], b[0], b[1], b[2]);
    Split4 s;
#pragma unroll
    for (int i = 0; i < 3; ++i) s.p[i] = u32x2_t{a[i], b[i]};
    return s;
}

template <bool LIMIT = false>
__device__ __forceinline__ Split8 split8(f32x4_t u, f32x4_t v)
{
    uint32_t x[4][3];
    split2<LIMIT>(u[0], u[1], x[0][0], x[0][1], x[0][2]);
    split2<LIMIT>(u[2], u[3], x[1][0], x[1][1], x[1][2]);
    split2<LIMIT>(v[0], v[1], x[2][0], x[2][1], x[2][2]);
    split2<LIMIT>(v[2], v[3], x[3][0], x[3][1], x[3][2]);
    Split8 s;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        s.p[i] = __builtin_bit_cast(bf16x8_t, u32x4_t{x[0][i], x[1][i], x[2][i], x[3][i]});
    return s;
}

__device__ __forceinline__ f32x4_t mfma32(bf16x8_t a, bf16x8_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// acc[k][n] += a[k] . b[n], the smallest products first. K and N together are
// the independent chains that follow each other on the matrix unit.
template <int K, int N>
__device__ __forceinline__ void product6(const bf16x8_t (&a)[K][3], const Split8* const (&b)[N], f32x4_t* const (&acc)[K][N])
{
    constexpr int ia[6] = {2, 0, 1, 1, 0, 0}, ib[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int n = 0; n < N; ++n) *acc[k][n] = mfma32(a[k][ia[i]], b[n]->p[ib[i]], *acc[k][n]);
}

// ND tiles of 16 cover a head; scores take KS steps of 32 of it. A tile in LDS
// has [array][piece][row][RS], with a row's groups of eight elements (16 bytes)
// exchanged by its number (attn_image_place), so that neither the 16-byte reads
// of sixteen rows (scores) nor the transposing reads of eight (results) meet in
// a bank. With rows of RS + 8 in plain order the latter took twice as long: 384
// us of 2 x 16 x 2,048 x 4,096 x 64 forward for 366, 783 by keys for 675.
template <int ND>
struct Heads {
    static constexpr int KS = (ND + 1) / 2, RS = 32 * KS;
};

// A wave's own row as the B operand of scores; not `valid`: zeros.
template <int ND>
__device__ __forceinline__ void load_own(Split8 (&f)[Heads<ND>::KS], const float* row, bool valid, int h, int dim)
{
#pragma unroll
    for (int c = 0; c < Heads<ND>::KS; ++c)
        f[c] = valid ? split8<true>(load4(row, 32 * c + 8 * h, dim), load4(row, 32 * c + 8 * h + 4, dim))
                     : split8(f32x4_t{}, f32x4_t{});
}

// The A operands of a step: of the two tiles of 16 rows (scores), or of two
// tiles of d (results).
struct Step {
    bf16x8_t a[2][3];
};

// AHEAD: the next step's operands are requested before the present step's
// products begin, which then hide the reads; for passes whose registers hold
// two steps. (Matrix instructions and reads of LDS keep their order across
// this; arithmetic, memory and LDS writes pass.)
template <bool AHEAD>
__device__ __forceinline__ void keep_order()
{
    if constexpr (AHEAD) __builtin_amdgcn_sched_barrier(0x2 | 0x4 | 0x10 | 0x200);
}

// acc[t][n] += (streamed rows 16 t .. of `tile`) . own[n]; PS: elements of a
// piece
template <int ND, int PS, bool AHEAD, int NT>
__device__ __forceinline__ void scores(const uint16_t* tile, int m, int h, const Split8 (&own)[NT][Heads<ND>::KS],
                                       f32x4_t (&acc)[2][NT])
{
    constexpr int RS = Heads<ND>::RS, KS = Heads<ND>::KS;
    const uint16_t* const at = tile + m * RS;
    const int place = 8 * (h ^ attn_image_place(KS, m));
    f32x4_t* to[2][NT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) to[t][n] = &acc[t][n];
    const auto load = [&](int c, Step& s) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 3; ++i) s.a[t][i] = *reinterpret_cast<const bf16x8_t*>(at + (place ^ 32 * c) + i * PS + 16 * t * RS);
    };
    Step step[2];
    if (AHEAD) load(0, step[0]);
#pragma unroll
    for (int c = 0; c < KS; ++c) {
        if (!AHEAD) load(c, step[c & 1]);
        if (AHEAD && c + 1 < KS) load(c + 1, step[(c + 1) & 1]);
        keep_order<AHEAD>();
        const Split8* b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) b[n] = &own[n][c];
        product6<2, NT>(step[c & 1].a, b, to);
    }
}

// acc[n] += (the 32 streamed rows at `tile`)^T . w[n], w from two score tiles
template <int ND, int PS, bool AHEAD, int NT>
__device__ __forceinline__ void results(const uint16_t* tile, int m, int h, const f32x4_t (&x)[2][NT], f32x4_t (&acc)[NT][ND])
{
    typedef __attribute__((address_space(3))) i16x4_t lds_t;
    constexpr int RS = Heads<ND>::RS, STEPS = (ND + 1) / 2;
    const int row = 4 * h + (m >> 2), place = 8 * ((m >> 1 & 1) ^ attn_image_place(Heads<ND>::KS, row));
    const uint16_t* const at = tile + row * RS + 4 * (m & 1);
    const auto load = [&](int p, Step& s) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (2 * p + t >= ND) continue;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const uint16_t* const from = at + (place ^ 16 * (2 * p + t)) + i * PS;
                const i16x4_t u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)from);
                const i16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(from + 16 * RS));
                s.a[t][i] = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        }
    };
    Step step[2];
    if (AHEAD) load(0, step[0]);
    Split8 w[NT];
    const Split8* b[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        w[n] = split8(x[0][n], x[1][n]);
        b[n] = &w[n];
    }
#pragma unroll
    for (int p = 0; p < STEPS; ++p) {
        if (!AHEAD) load(p, step[p & 1]);
        if (AHEAD && p + 1 < STEPS) load(p + 1, step[(p + 1) & 1]);
        keep_order<AHEAD>();
        if (2 * p + 1 < ND) {
            f32x4_t* to[2][NT];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n) to[t][n] = &acc[n][2 * p + t];
            product6<2, NT>(step[p & 1].a, b, to);
        } else {
            f32x4_t* to[1][NT];
            const bf16x8_t one[1][3] = {{step[p & 1].a[0][0], step[p & 1].a[0][1], step[p & 1].a[0][2]}};
#pragma unroll
            for (int n = 0; n < NT; ++n) to[0][n] = &acc[n][2 * p < ND ? 2 * p : 0];
            product6<1, NT>(one, b, to);
        }
    }
}

// A result's column to a row of `dim` floats, times f.
template <int ND>
__device__ __forceinline__ void store_own(const f32x4_t (&acc)[ND], float f, float* row, int h, int dim)
{
#pragma unroll
    for (int t = 0; t < ND; ++t) store4(row, 16 * t + 4 * h, dim, acc[t] * f);
}

// A row's product with another, both in memory, in all of its lanes.
template <int ND>
__device__ __forceinline__ float row_dot(const float* x, const float* y, int h, int dim)
{
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < ND; ++t) {
        const f32x4_t u = load4(x, 16 * t + 4 * h, dim), v = load4(y, 16 * t + 4 * h, dim);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = __builtin_fmaf(u[e], v[e], sum);
    }
    return column_sum(sum);
}

template <int ND, int NT>
__device__ __forceinline__ void clear(f32x4_t (&acc)[NT][ND])
{
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < ND; ++t) acc[n][t] = f32x4_t{};
}

// Waves that share a SIMD would go through the same loop side by side, all at
// its matrix products, then all at its exponentials and splits. Every second one
// is given way to, so that it is ahead by a phase. us without and with: 7 x 6 heads
// of 257 x 777 x 80, ragged, forward 37.7 and 36.4, backward 99.4 and 98.1, second
// order 288 and 283; no difference in long sequences (2 x 16 of 2,048 x 4,096 x 64 360
// and 362, 1,133 and 1,136, 3,581 and 3,577; 2 x 16 of 1,000 x 2,048 x 128 alike).
__device__ __forceinline__ void stagger()
{
    constexpr int kHwId = 4, kWaveSlotBits = 4;   // HW_REG_HW_ID: the wave's slot in its SIMD
    if (__builtin_amdgcn_s_getreg(kHwId | (kWaveSlotBits - 1) << 11) & 1) __builtin_amdgcn_s_setprio(2);
}

// ---- the streamed side ------------------------------------------------------------
//
// N arrays of rows and X numbers per row, 32 at a time, from one of two
// sources. Where several teams stream the same side, it is split beforehand
// into images of the tiles in LDS (emu_attn_planes.hip), which are copied there
// directly, the next one while the present one is used. Otherwise the team
// reads the arrays themselves and splits them on the way; where registers
// allow, the next tile is requested before the present one is used.
// Two buffers in LDS, so that one barrier a tile does, where they leave room
// for the RESIDENT workgroups that registers hold, or one buffer alone does not.

constexpr int kStreamRows = kAttnTile;

// An array as a thread reads it: a tile's rows begin at base + first row / 32
// * tile floats, the thread's there at offset + e * step.
struct StreamRows {
    const float* base;       // null: zeros
    int64_t tile, step;
    int offset;
};

constexpr int kTeam = 4;   // waves that share a streamed tile

template <int ND, int N, int X, bool KEYS, bool IMAGES, int RESIDENT>
struct Stream {
    using T = Team<kTeam>;
    static constexpr int RS = Heads<ND>::RS, kPiece = kStreamRows * RS, kArray = 3 * kPiece;
    // threads along a row (a power of two), a thread's rows and the distance between them
    static constexpr int kQuads = Heads<ND>::KS == 3 ? 32 : 8 * Heads<ND>::KS, kStep = T::kThreads / kQuads < kStreamRows ? T::kThreads / kQuads : kStreamRows;
    static constexpr int kEach = kStreamRows / kStep;
    static constexpr int kArrays = IMAGES ? (int)attn_image_bytes(16 * ND, N) : N * kArray * 2;
    static constexpr int kBytes = kArrays + X * kStreamRows * 4;
    static constexpr bool kAhead = N * kEach <= 8;
    static constexpr int kLds = 160 * 1024, kShare = kLds / RESIDENT;   // a compute unit's, a team's
    static constexpr bool kTwo = (IMAGES || kAhead) && (2 * kBytes <= kShare || (IMAGES && kBytes > kShare && 2 * kBytes <= kLds));
    static constexpr int kBuffers = kTwo ? 2 : 1;
    static_assert(kBytes % 16 == 0, "buffers stay aligned");
    static_assert(RS == attn_image_row(16 * ND), "images are tiles as they lie in LDS");

    char* base;
    int turn = 0;

    // The tiles lo .. hi of `images`, which hold the side's tiles in order.
    template <class Q, class F>
    __device__ __forceinline__ void run_images(const char* images, int64_t lo, int64_t hi, Q&& number, F&& f)
    {
        float numbers[X];
        const auto request = [&](int64_t first) {
            // (before the copies, which are waited for together with them)
            if (T::thread() < kStreamRows) number(first, numbers);
            char* const buffer = base + (kBuffers == 2 ? (turn ^ 1) * kBytes : 0);
            const uint32_t to = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)buffer;
            const char* const from = images + (first / kStreamRows) * kArrays;
#pragma unroll
            for (int c = 0; c < (kArrays / 1024 + kTeam - 1) / kTeam; ++c) {
                const int chunk = c * kTeam + T::wave();
                if (chunk < kArrays / 1024) copy16_to_lds(to + chunk * 1024, from, (uint32_t)(chunk * 1024 + (threadIdx.x & 63) * 16));
            }
        };
        if (kBuffers == 2 && lo < hi) {
            T::sync();   // (a previous piece's last tile has been read)
            request(lo);
        }
        for (int64_t first = lo; first < hi; first += kStreamRows) {
            if (kBuffers == 1) {
                T::sync();   // the previous tile has been read
                request(first);
            }
            wait_vmcnt<0>();
            if (kBuffers == 2) turn ^= 1;
            char* const buffer = base + (kBuffers == 2 ? turn * kBytes : 0);
            float* const nums = reinterpret_cast<float*>(buffer + kArrays);
            if (T::thread() < kStreamRows) {
#pragma unroll
                for (int i = 0; i < X; ++i) nums[i * kStreamRows + T::thread()] = numbers[i];
            }
            T::sync();
            if (kBuffers == 2 && first + kStreamRows < hi) request(first + kStreamRows);
            if (!(KEYS && __all(nums[threadIdx.x & 31] == minus_inf())))
                f(first, reinterpret_cast<const uint16_t*>(buffer), const_cast<const float*>(nums));
        }
    }

    struct Tile {
        f32x4_t v[kEach];
    };

    // Once: what lies past the heads' width is zero and stays so.
    __device__ __forceinline__ void clear()
    {
        if (IMAGES) return;
        for (int i = T::thread(); i < kBuffers * kBytes / 16; i += T::kThreads) reinterpret_cast<u32x4_t*>(base)[i] = u32x4_t{};
        T::sync();
    }

    static_assert(kStep * kEach == kStreamRows && T::kThreads <= kQuads * kStreamRows, "every thread has whole quads of rows");
    static __device__ __forceinline__ int row() { return T::thread() / kQuads; }
    static __device__ __forceinline__ int col() { return T::thread() % kQuads * 4; }

    // f(first row, arrays, numbers) for the tiles of lo .. hi (lo a multiple of
    // 32): array i at arrays + i kArray, its number x of row r at numbers + x
    // kStreamRows + r.
    // rows(i): array i's StreamRows; even: they hold for whole tiles (else,
    // and in the last, cut tile, where(i, row) is the row's address).
    // number(first, numbers): those of row first + thread, < 32.
    // KEYS: number 0 is a key's term; keys that take no part (dropped(row), if
    // some are) are zeros, and a tile of such keys alone is left out. (The
    // others' scores of a row are then finite plus -infinity, or as little as
    // the row's own infinities leave of any score.)
    template <class R, class P, class D, class Q, class F>
    __device__ __forceinline__ void run(int64_t lo, int64_t hi, int dim, bool even, R&& rows, P&& where, bool some,
                                        D&& dropped, Q&& number, F&& f)
    {
        Tile tiles[N];
        float numbers[X];
        uint32_t drop = 0;   // bit e: the thread's row e
        even = even && dim % 4 == 0;
        const bool has = col() < dim;
        const auto fetch = [&](int i, int64_t first) {
            Tile& t = tiles[i];
            const StreamRows r = rows(i);
            if (even && first + kStreamRows <= hi) {
                if (r.base == nullptr || !has) return;   // (zeros since clear())
                const char* from = reinterpret_cast<const char*>(r.base + (first >> 5) * r.tile);
                const uint32_t at = (uint32_t)(r.offset + col()) * 4u;
#pragma unroll
                for (int e = 0; e < kEach; ++e) t.v[e] = *reinterpret_cast<const f32x4u_t*>(from + e * r.step * 4 + at);
            } else if (r.base != nullptr) {
                // (float by float, clamped to what is there)
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const int64_t at = first + row() + e * kStep;
                    const float* const p = where(i, at < hi ? at : hi - 1);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const bool there = at < hi && col() + x < dim;
                        const float y = p[col() + x < dim ? col() + x : dim - 1];
                        t.v[e][x] = there ? y : 0.0f;
                    }
                }
            }
        };
        const auto request = [&](int64_t first) {
            if constexpr (kAhead) {
#pragma unroll
                for (int i = 0; i < N; ++i) fetch(i, first);
            }
            if (T::thread() < kStreamRows) number(first, numbers);
            if (KEYS && some) {
                drop = 0;
#pragma unroll
                for (int e = 0; e < kEach; ++e) drop |= dropped(first + row() + e * kStep) ? 1u << e : 0u;
            }
        };
        // (the first turn only requests)
        for (int64_t first = lo - kStreamRows; first < hi; first += kStreamRows) {
            const bool here = first >= lo;
            char* buffer = base;
            if (here) {
                if (kBuffers == 1) T::sync();   // the previous tile has been read
                if (kBuffers == 2) buffer += (turn ^= 1) * kBytes;
                uint16_t* const arrays = reinterpret_cast<uint16_t*>(buffer);
                if constexpr (!kAhead) {
#pragma unroll
                    for (int i = 0; i < N; ++i) fetch(i, first);
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (!has || rows(i).base == nullptr) continue;
                    if (KEYS && some && __any(drop != 0)) {
#pragma unroll
                        for (int e = 0; e < kEach; ++e)
                            if (drop >> e & 1) tiles[i].v[e] = f32x4_t{};
                    }
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        const Split4 s = split4(tiles[i].v[e]);
#pragma unroll
                        for (int p = 0; p < 3; ++p) {
                            const int r = row() + e * kStep;
                            uint16_t* const to = arrays + i * kArray + p * kPiece + r * RS;
                            *reinterpret_cast<u32x2_t*>(to + 8 * (col() / 8 ^ attn_image_place(Heads<ND>::KS, r)) + col() % 8) = s.p[p];
                        }
                    }
                }
                if (T::thread() < kStreamRows) {
                    float* const nums = reinterpret_cast<float*>(buffer + N * kArray * 2);
#pragma unroll
                    for (int i = 0; i < X; ++i) nums[i * kStreamRows + T::thread()] = numbers[i];
                }
                T::sync();
            }
            if (first + kStreamRows < hi) request(first + kStreamRows);
            const float* const nums = reinterpret_cast<const float*>(buffer + N * kArray * 2);
            // (a tile of keys that take no part adds nothing, whatever the rows hold)
            if (here && !(KEYS && some && __all(nums[threadIdx.x & 31] == minus_inf())))
                f(first, reinterpret_cast<const uint16_t*>(buffer), nums);
        }
    }

    // The keys' side: arrays of the keys' shape.
    template <class Q, class F, class... A>
    __device__ __forceinline__ void run_keys(const AttnArgs& a, const Piece& at, const char* images, int64_t lo, int64_t hi,
                                             Q&& number, F&& f, const A&... arrays)
    {
        if constexpr (IMAGES) {
            const int64_t tiles = (a.keys + kStreamRows - 1) / kStreamRows;
            return run_images(images + ((int64_t)at.b * a.kv_heads + at.g) * tiles * kArrays, lo, hi, number, f);
        }
        const emu_heads_t of[N] = {arrays...};
        bool even = true;
#pragma unroll
        for (int i = 0; i < N; ++i) even = even && fits(of[i].token);
        run(
            lo, hi, a.dim, even,
            [&](int i) {
                const emu_heads_t& t = of[i];
                return StreamRows{t.data != nullptr ? key_ptr(t, at.b, at.g, 0) : nullptr, kStreamRows * t.token, kStep * t.token,
                                  row() * (int)t.token};
            },
            [&](int i, int64_t row) { return key_ptr(of[i], at.b, at.g, row); }, a.bias != nullptr || a.mask != nullptr,
            [&](int64_t row) { return key_term(a, at.b, (int)row, (int)hi) == minus_inf(); }, number, f);
    }

    // The rows' side: arrays of the queries' shape.
    template <class Q, class F, class... A>
    __device__ __forceinline__ void run_rows(const AttnArgs& a, const Piece& at, const char* images, int64_t lo, int64_t hi,
                                             Q&& number, F&& f, const A&... arrays)
    {
        if constexpr (IMAGES) {
            const int64_t tiles = (a.rows + kStreamRows - 1) / kStreamRows;
            return run_images(images + ((int64_t)at.b * a.kv_heads + at.g) * tiles * kArrays, lo, hi, number, f);
        }
        const emu_heads_t of[N] = {arrays...};
        // (a thread's rows are a whole number of queries apart)
        bool even = a.share <= kStep && kStep % a.share == 0;
#pragma unroll
        for (int i = 0; i < N; ++i) even = even && fits(of[i].token) && fits(of[i].head);
        const RowAt mine = row_at(a, 0, row());   // (query and head of a tile's row)
        run(
            lo, hi, a.dim, even,
            [&](int i) {
                const emu_heads_t& t = of[i];
                return StreamRows{t.data != nullptr ? row_ptr(t, at.b, RowAt{0, at.g * a.share}) : nullptr,
                                  kStreamRows / a.share * t.token, kStep / a.share * t.token,
                                  mine.query * (int)t.token + mine.head * (int)t.head};
            },
            [&](int i, int64_t row) { return row_ptr(of[i], at.b, row_at(a, at.g, row)); }, false,
            [](int64_t) { return false; }, number, f);
    }

    // 32 strides of tokens and of heads in 32 bits of bytes, none backwards
    static __device__ __forceinline__ bool fits(int64_t stride) { return stride >= 0 && stride < ((int64_t)1 << 24); }
};

// The terms of a lane's keys: 0 .. 3 of the first 16 at its group, then of the
// second.
struct Terms {
    f32x4_t of[2];
    __device__ __forceinline__ Terms(const float* term, int h)
    {
        of[0] = *reinterpret_cast<const f32x4_t*>(term + 4 * h);
        of[1] = *reinterpret_cast<const f32x4_t*>(term + 16 + 4 * h);
    }
};

// f.template operator()<ND, NT, IMAGES>() for a head and plan.
template <AttnPass PASS, class F>
inline void with_shape(int dim, const AttnPlan& p, F&& f)
{
    const auto tiles = [&]<int ND>() {
        constexpr int NT = attn_tiles(PASS, 16 * ND);
        if (p.images) return f.template operator()<ND, NT, true>();
        if constexpr (NT == 2) {
            if (p.tiles == 2) return f.template operator()<ND, 2, false>();
        }
        return f.template operator()<ND, 1, false>();
    };
    if (dim <= 16)
        tiles.template operator()<1>();
    else if (dim <= 32)
        tiles.template operator()<2>();
    else if (dim <= 48)
        tiles.template operator()<3>();
    else if (dim <= 64)
        tiles.template operator()<4>();
    else if (dim <= 80)
        tiles.template operator()<5>();
    else if (dim <= 96)
        tiles.template operator()<6>();
    else
        tiles.template operator()<8>();
}

}  // namespace emu
