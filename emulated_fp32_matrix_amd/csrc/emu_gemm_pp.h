// The two-group form of the emulated-FP32 GEMM (its description is with the
// kernel below; the method and the other kernels are in emu_gemm_bf16.hip),
// shared by the plain GEMM and the operators that add more to its epilogue
// (gfx950 only).
#pragma once

#include "emu_block_device.h"
#include "emu_block_launch.h"
#include "emu_tile.h"
#include "emu_walk.h"

namespace emu {

// What is done with a finished output tile.
enum { EPI_PLAIN = 0, EPI_ACT = 1, EPI_GATED = 2 };

// Row of the gated projection's weight (2 F rows: gate, then up) behind row r
// of its B planes' 128-row tile tr, or -1: every 32 rows hold 16 gates and
// the 16 up rows of the same columns of C.
__host__ __device__ constexpr int64_t gated_plane_row(int64_t tr, int r, int64_t F)
{
    const int64_t h = tr * 64 + (r >> 5) * 16 + (r & 15);
    return h >= F ? -1 : (r & 16) == 0 ? h : F + h;
}

constexpr int PS = TILE * LDS_ROW; // elements per plane of an LDS tile

// Plane rows carry no padding.  Instead the four 16-byte chunks of row r
// (k = 8c .. 8c+7 in chunk c) are stored in the order c ^ plane_swz(r), which
// depends on r % 16 only.  The permutation was chosen by timing the two LDS
// patterns of the kernel on gfx950 with candidate permutations: the MFMA
// fragment reads (lane l: row l % 32, chunk 2 ks + l / 32, 16 bytes) run at
// 464 B/ns per CU with this one, against 433 with rows padded to 80 bytes
// and 303 with ((r >> 1) ^ (r >> 3)) & 3; the split's 8-byte writes run at
// 182 against 153 padded.  It also saves a fifth of every plane's LDS space
// and of the B chunks' load volume.
__host__ __device__ constexpr int plane_swz(int r) { return (r >> 2) & 3; }
// Element offset of (row r, k) within one plane.
__host__ __device__ constexpr int plane_elem(int r, int k)
{
    return r * LDS_ROW + ((((k >> 3) ^ plane_swz(r)) << 3) | (k & 7));
}

__host__ __device__ constexpr int64_t chunk_elems(int np) { return (int64_t)np * PS; }

namespace {

// The kernel's BlockEpilogue argument, read from its argument segment where
// the epilogue begins: held in scalar registers through the main loop
// instead, its 18 words spilled 40 of them, and those into vector registers.
template <class E>
__device__ __forceinline__ E reload_epilogue(const E& e)
{
#ifndef __HIP_DEVICE_COMPILE__
    return e;   // (the host pass only parses this)
#else
    typedef const __attribute__((address_space(4))) char* kernarg_t;
    constexpr int at = (sizeof(Params) + 7) / 8 * 8 + sizeof(void*);   // (Params, Wb, epilogue)
    static_assert(alignof(E) == 8, "arguments of 8-byte alignment");
    kernarg_t k = (kernarg_t)__builtin_amdgcn_kernarg_segment_ptr() + at;
    asm volatile("" : "+s"(k));   // (not hoisted out of the loop)
    return *reinterpret_cast<const __attribute__((address_space(4))) E*>(k);
#endif
}

// ---------------------------------------------------------------------------
// Ping-pong form of the GEMM kernel for a k-contiguous FP32 op(A) (split in
// the kernel).  The 8 waves form two groups of four, one wave of each group
// per SIMD; group g owns rows 64g..64g+63 of the 128x128 tile, each of its
// waves a 64x32 block (two 32x32 MFMA tiles).  Each group alternates two
// kinds of phase, each closed by a workgroup barrier:
//   U(s): reads the group's FP32 A rows of step s+1 from staging, then
//         (while those reads are in flight) runs the epilogue of the tile
//         that ended at step s-1 and issues the direct loads of its half of
//         a B chunk (group 0: step s+1, group 1: step s+2) and of its A rows
//         of step s+2, then splits the step s+1 rows into the other plane
//         buffer;
//   M(s): the MFMAs of step s, then the scalar bookkeeping (advancing the
//         step cursors, precomputing addresses) for the next U phase, and
//         the wait for the group's half of B loaded in U(s).
// Group 1 starts one phase late, so U of one group runs beside M of the
// other: on every SIMD one wave keeps the matrix unit busy while the other
// does the vector, LDS and memory work.  Since a wave issues one instruction
// at a time, scalar work costs issue slots in a U phase but fills idle ones
// between the MFMAs of an M phase, which is where it is placed.  An M
// phase's fragment reads run one group of MFMAs ahead of their use, the
// first group's (A and B) before the barrier.  The split's LDS writes are only waited
// for at the end of the next M phase, and each thread splits exactly the A
// elements it loaded itself, so its own load-counter wait publishes them to
// itself.
// LDS: two plane buffers for A (each group touches only its own rows),
// three B chunk buffers (chunks s-1 .. s+1 while group 0 loads its half of
// s+1, s .. s+2 while group 1 loads its half of s+2), two FP32
// staging buffers (step s+2 overwrites step s, split in U(s-1)): 152 KB
// with three planes.
// ---------------------------------------------------------------------------

// GENERAL: the epilogue reads C (beta != 0) or adds a bias; the plain
// instantiation (C = alpha t) carries neither path, which saves it SGPR
// spills and registers in the loop (1.6 % on the 552,960-row stack).
// TH: rows of an output tile, 128 or 64 (the 64-row tiles give shapes with
// few tiles more of them; each group then owns 32 rows).
// EPI: what is done with a finished tile (EPI_PLAIN: C = alpha t + beta C +
// bias; EPI_ACT and EPI_GATED: see BlockEpilogue, the kernel's last argument
// then).
template <int NB, bool SPLIT, bool GENERAL, int TH, int EPI, class... Epi>
__global__ __launch_bounds__(512, 1) void gemm_bf16_pp_kernel(Params p, const uint16_t* __restrict__ Wb, Epi... finish)
{
    static_assert(EPI == EPI_PLAIN ? sizeof...(Epi) == 0 : !GENERAL && sizeof...(Epi) == 1,
                  "the block operators' epilogue takes its description, the plain one none");
    static_assert(!(SPLIT && GENERAL), "a split launch reads beta and the bias at run time");
    static_assert(TH == 128 || TH == 64, "output tiles of 128 or 64 rows");
    constexpr int NP = NB >= 3 ? 3 : NB;
    constexpr int CHUNK_BYTES = (int)chunk_elems(NP) * 2;
    constexpr int GT = 256;                                // threads per group
    constexpr int GROWS = TH / 2;                          // A rows per group
    constexpr int PSA = TH * LDS_ROW;                      // elements per A plane
    constexpr int B_ROUNDS = CHUNK_BYTES / (GT * 16);      // 4 KB rounds per B chunk
    constexpr int B_HALF = B_ROUNDS / 2;                   // rounds each group copies
    constexpr int A_ROUNDS = GROWS * BK * 4 / (GT * 16);   // 16-byte loads per thread
    constexpr int TM = GROWS / 32;                         // 32x32 MFMA blocks per wave
    static_assert(A_ROUNDS == TM && GROWS == TM * 32, "thread t splits rows t/8 + 32r of its group");
    static_assert(B_ROUNDS * GT * 16 == CHUNK_BYTES && B_HALF * 2 == B_ROUNDS, "B chunk in whole half rounds");
    __shared__ __attribute__((aligned(16))) uint16_t smA[2][NP * PSA];
    __shared__ __attribute__((aligned(16))) uint16_t smB[3][chunk_elems(NP)];
    __shared__ __attribute__((aligned(16))) float stage[2][TH * BK];

    const int G = gridDim.x;
    const int slot = xcd_position(blockIdx.x, G);
    // Items: tiles 0 .. split_from-1 whole, then (SPLIT) the ksplit K
    // segments of each of the other tiles; this workgroup's are slot, slot +
    // G, ...  (split_from is 0, every tile split, or a multiple of G: whole
    // rounds of whole tiles, then the last round's tiles split.)
    const int nsplit = SPLIT ? p.ntiles - p.split_from : 0;
    const int nitems = SPLIT ? p.split_from + nsplit * p.ksplit : p.ntiles;
    const int my_items = (nitems - slot + G - 1) / G;
    const int my_whole = SPLIT ? (slot < p.split_from ? (p.split_from - slot + G - 1) / G : 0) : my_items;
    const int total = my_whole * p.nk + (my_items - my_whole) * p.nk_item;

    WalkConst wc;
    const int gtile = G % p.ntiles;   // tiles added per advance
    wc.nk = p.nk;
    wc.nk_item = p.nk_item;
    wc.th = TH;
    wc.G = G;
    wc.split_from = SPLIT ? p.split_from : p.ntiles;
    wc.nsplit = nsplit > 0 ? nsplit : 1;
    wc.tiles_n = p.tiles_n;
    wc.gtn = gtile % p.tiles_n;
    wc.gm = (int64_t)(gtile / p.tiles_n) * TH;
    wc.tail_k = (int)(p.K - (int64_t)(p.nk - 1) * BK);
    wc.M = p.M;
    wc.lda = p.lda;

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);  // wave-uniform
    const int grp = wave >> 2;
    const int gw = wave & 3;          // wave within the group = its 32-column block
    const int gt = t & (GT - 1);
    const int frag_row = lane & 31;
    const int frag_k = (lane >> 5) * 8;

    // Thread gt of group g loads and splits rows GROWS g + gt/8 + 32r (r <
    // A_ROUNDS), k = 4(gt%8) .. +3 of each step's FP32 A tile.
    const int srow0 = GROWS * grp + (gt >> 3);
    const int skc = (gt & 7) * 4;
    uint32_t a_off[A_ROUNDS];
#pragma unroll
    for (int r = 0; r < A_ROUNDS; ++r)
        a_off[r] = (uint32_t)(((int64_t)(srow0 + 32 * r) * p.lda + skc) * 4);

    // Round r (of A_ROUNDS) of the group's FP32 A rows of step w into
    // staging buffer sb: staging is [TH][32] floats, this wave's 64 lanes
    // fill 1 KB at row GROWS g + 8 gw + 32 r.
    auto copy_a32_round = [&](const Walk& w, int sb, int r) __attribute__((always_inline)) {
        const float* base = p.A + w.arow + (int64_t)w.kt * BK;
        const uint32_t dst = lds_offset(stage[sb]) + GROWS * BK * 4 * grp + 1024 * gw;
        uint32_t off = a_off[r];
        if (w.rows != TH || w.kvalid != BK) {
            // rows past M re-read the tile's last row, k past K column 0
            // (both masked when split)
            const int row = srow0 + 32 * r;
            const int64_t rr = row < w.rows ? row : w.rows - 1;
            const int kk = skc < w.kvalid ? skc : 0;
            off = (uint32_t)((rr * p.lda + kk) * 4);
        }
        copy16_to_lds(dst + 4096 * r, base, off);
    };
    auto copy_a32 = [&](const Walk& w, int sb) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < A_ROUNDS; ++r) copy_a32_round(w, sb, r);
    };
    // This group's half of the B chunk of step w into buffer bb: rounds
    // B_HALF g .. B_HALF g + B_HALF - 1, round r the 4 KB at 4096 r, this
    // wave's 1 KB piece of it at 4096 r + 1024 gw.
    auto copy_b_half = [&](const Walk& w, int bb) __attribute__((always_inline)) {
        const char* src = reinterpret_cast<const char*>(Wb + ((int64_t)w.tn * p.nk + w.kt) * chunk_elems(NP));
        const uint32_t dst = lds_offset(smB[bb]);
#pragma unroll
        for (int j = 0; j < B_HALF; ++j) {
            const int byte0 = ((grp * B_HALF + j) * GT + gw * 64) * 16;
            copy16_to_lds(dst + byte0, src + byte0, (uint32_t)lane * 16);
        }
    };
    // The split of the group's rows of one step, in two parts: load_rows
    // reads the thread's FP32 values from staging buffer sb (on edge tiles,
    // elements outside op(A) selected to zero); split_rows splits them into
    // plane buffer ab.
    auto load_rows = [&](const Walk& w, int sb, f32x4_t (&v)[A_ROUNDS]) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < A_ROUNDS; ++q)
            v[q] = *reinterpret_cast<const f32x4_t*>(&stage[sb][(srow0 + 32 * q) * BK + skc]);
        if (w.rows != TH || w.kvalid != BK) {
#pragma unroll
            for (int q = 0; q < A_ROUNDS; ++q) {
                const bool rok = srow0 + 32 * q < w.rows;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[q][e] = (rok && skc + e < w.kvalid) ? v[q][e] : 0.0f;
            }
        }
    };
    const int split_off = plane_elem(srow0, skc);   // rows 32 apart share the chunk order
    auto split_rows = [&](const f32x4_t (&v)[A_ROUNDS], int ab) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < A_ROUNDS; ++q) {
            uint32_t w0[NP], w1[NP];
            split_pieces<NP>(v[q][0], v[q][1], w0);
            split_pieces<NP>(v[q][2], v[q][3], w1);
            uint16_t* dst = smA[ab] + split_off + 32 * q * LDS_ROW;
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) *reinterpret_cast<u32x2_t*>(dst + pl * PSA) = u32x2_t{w0[pl], w1[pl]};
        }
    };

    // Accumulators: cleared here and after each tile's epilogue.
    f32x16_t acc[TM][NB];
    auto clear_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[i][b] = zero_acc();
    };
    clear_acc();

    // Operand fragments of k-half ks: this wave's B columns (all planes) in
    // B buffer bb and its A rows of plane u in plane buffer ab.  Fragment
    // rows start at multiples of 32, so the lane's offset within a plane is
    // frag_off0 (ks = 0) or frag_off1 (ks = 1) past the first row's.
    const int frag_off0 = plane_elem(frag_row, frag_k), frag_off1 = plane_elem(frag_row, 16 + frag_k);
    auto load_bfr = [&](int bb, int ks, bf16x8_t (&bfr)[NP]) __attribute__((always_inline)) {
#pragma unroll
        for (int pl = 0; pl < NP; ++pl)
            bfr[pl] = *reinterpret_cast<const bf16x8_t*>(smB[bb] + pl * PS + gw * 32 * LDS_ROW +
                                                         (ks ? frag_off1 : frag_off0));
    };
    auto load_afr = [&](int ab, int ks, int u, bf16x8_t (&af)[TM]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            af[i] = *reinterpret_cast<const bf16x8_t*>(smA[ab] + u * PSA + (grp * GROWS + i * 32) * LDS_ROW +
                                                       (ks ? frag_off1 : frag_off0));
    };
    // The MFMAs of one plane u of A against all planes of B (fragments
    // already in registers), smallest band first.
    auto mfma_u = [&](int u, const bf16x8_t (&bfr)[NP], const bf16x8_t (&af)[TM]) __attribute__((always_inline)) {
#pragma unroll
        for (int v = NP - 1; v >= 0; --v) {
            if (u + v < NB) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    // B operand first: lane l then holds row l%32 of the
                    // 32x32 block and four consecutive columns per register
                    // group, for 16-byte stores.
                    acc[i][u + v] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bfr[v], af[i], acc[i][u + v], 0, 0, 0);
            }
        }
    };

    // Epilogue of this wave's block of the item at w: bands recombined
    // smallest first into t, then C = alpha t + beta C + bias, or for a K
    // segment of a split tile (part) t itself into the segment's slot of the
    // workspace (TH x 128 floats, rows of 128).  Lane l holds, per 32x32
    // block and register group q, row l%32 and columns 8q + 4(l/32) .. +3:
    // one 16-byte buffer store each, rows outside C given an out-of-range
    // offset.  Tiles that cross column N, or a destination without 16-byte
    // rows, store element by element.  SCALE: alpha != 1.
    // In a split launch one copy serves both kinds of item, its destination
    // and scalars chosen at run time (a part: alpha 1, which is exact, no
    // beta, no bias; a whole tile takes them here, a split one in the
    // reduction).
    auto epilogue = [&]<bool SCALE>(const TilePos& w) __attribute__((always_inline)) {
        const int64_t n0 = (int64_t)w.tn * TILE;
        int64_t ldd = p.ldc;
        float* dst = p.C + w.m0 * p.ldc + n0;
        float alpha = p.alpha;
        float beta = GENERAL || SPLIT ? p.beta : 0.0f;
        const float* bias = GENERAL || SPLIT ? p.bias : nullptr;
        bool part = false;
        if constexpr (SPLIT) {
            part = w.part != 0;
            if (part) {
                ldd = TILE;
                dst = p.wsC + (int64_t)w.widx * (TH * TILE);
                alpha = 1.0f;
                beta = 0.0f;
                bias = nullptr;
            }
        }
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(dst, (short)0, 0x7FFFFFFF, 0x00020000);
        const int64_t cl = p.N - n0;
        const int cols_left = cl < TILE ? (int)cl : TILE;
        // vec_b / vec_ws carry the destination's (and the bias') alignment
        const bool vec_c = (part ? p.vec_ws : p.vec_b) != 0 && cols_left == TILE;
        const int ldd4 = (int)ldd * 4;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int row = grp * GROWS + i * 32 + (lane & 31);
            const bool row_ok = row < w.rows;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = gw * 32 + 8 * q + 4 * (lane >> 5);
                f32x4_t out;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 4 * q + e;
                    float sum = acc[i][NB - 1][r];
#pragma unroll
                    for (int b = NB - 2; b >= 0; --b) sum = __builtin_fmaf(sum, 0.00390625f, acc[i][b][r]);
                    out[e] = SCALE ? alpha * sum : sum;
                }
                if (vec_c) {
                    const int off = row_ok ? row * ldd4 + col * 4 : (int)0x80000000;
                    if (beta != 0.0f) {
                        const f32x4_t old = __builtin_bit_cast(
                            f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, 0));
#pragma unroll
                        for (int e = 0; e < 4; ++e) out[e] = __builtin_fmaf(beta, old[e], out[e]);
                    }
                    if (bias != nullptr) {
                        // The wave's 8 bias values of register group q sit at a
                        // wave-uniform address: read them with one scalar load
                        // (counted by lgkmcnt, so waiting for it never waits for
                        // the direct loads in flight) and pick this lane's four.
                        const i32x8_t bv = scalar_load8(bias + n0 + gw * 32 + 8 * q);
                        const bool upper = (lane >> 5) != 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // (opaque copies: otherwise the two selects fold into an
                            // index into bv and a chain of compares)
                            int lo = bv[e], hi = bv[4 + e];
                            asm("" : "+s"(lo));
                            asm("" : "+s"(hi));
                            out[e] = out[e] + __int_as_float(upper ? hi : lo);
                        }
                    }
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, out), rsrc, off, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (row_ok && col + e < cols_left) {
                            float* cp = dst + row * ldd + col + e;
                            float o = out[e];
                            if (beta != 0.0f) o = __builtin_fmaf(beta, *cp, o);
                            if (bias != nullptr) o = o + bias[n0 + col + e];
                            *cp = o;
                        }
                    }
                }
            }
        }
    };
    // Epilogue of the transformer-block operators: the bands recombined to t,
    // then z = t + bias, optionally written to Z, and C = act(z) + R
    // (EPI_ACT), or with t = [g | u] C = act(g) u (EPI_GATED).  The gated
    // planes hold 16 gate and the same 16 up columns in every 32 (see
    // gated_plane_row), so a lane's register groups 0, 1 are the gates of
    // its groups 2, 3: 64 columns of C per tile, the pairs in one lane.
    // The activation follows the recombination of a 32-row block, whose band
    // accumulators are free by then.  Residuals are requested before it.
    auto block_epilogue = [&](const TilePos& w, const BlockEpilogue& be) __attribute__((always_inline)) {
        constexpr int CW = EPI == EPI_GATED ? TILE / 2 : TILE;   // columns of C per tile
        const bool part = SPLIT && w.part != 0;
        const int64_t n0 = (int64_t)w.tn * CW;
        const int64_t cl = p.N - n0;
        const int cols_left = cl < CW ? (int)cl : CW;
        const bool full = part || (cols_left == CW && p.vec_b != 0);
        float* cbase = part ? p.wsC + (int64_t)w.widx * (TH * TILE) : be.C + w.m0 * be.ldc + n0;
        const int64_t ldc = part ? TILE : be.ldc;
        const float* rbase = be.R + w.m0 * be.ldr + n0;
        float* zbase = be.Z + w.m0 * be.ldz + n0;
        const bool has_z = be.Z != nullptr && !part;
        const bool has_r = EPI == EPI_ACT && be.R != nullptr && !part;
        auto rsrc = [](const float* q) __attribute__((always_inline)) {
            return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(q), (short)0, 0x7FFFFFFF, 0x00020000);
        };
        const int half4 = 4 * (lane >> 5);
        // every residual of the wave's rows is requested here: one memory
        // latency per tile
        f32x4_t res[EPI == EPI_ACT ? TM : 1][4];
        if constexpr (EPI == EPI_ACT) {
            if (has_r) {
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int row = grp * GROWS + i * 32 + (lane & 31);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int col = gw * 32 + 8 * q + half4;
                        if (full)
                            res[i][q] = __builtin_bit_cast(
                                f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                             rsrc(rbase), row < w.rows ? (row * (int)be.ldr + col) * 4 : (int)0x80000000, 0, 0));
                        else
                            res[i][q] = row < w.rows ? load4(rbase + row * be.ldr, col, cols_left) : f32x4_t{};
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int row = grp * GROWS + i * 32 + (lane & 31);
            const bool row_ok = row < w.rows;
            // column of C (or of the partial tile) of register group q
            auto col_of = [&](int q) __attribute__((always_inline)) {
                return EPI == EPI_GATED && !part ? gw * 16 + 8 * (q & 1) + half4 : gw * 32 + 8 * q + half4;
            };
            auto offset = [&](int64_t ld, int col) __attribute__((always_inline)) {
                return row_ok ? (row * (int)ld + col) * 4 : (int)0x80000000;
            };
            auto put = [&](float* base, int64_t ld, int col, f32x4_t v) __attribute__((always_inline)) {
                if (full)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rsrc(base), offset(ld, col), 0, 0);
                else if (row_ok)
                    store4(base + row * ld, col, cols_left, v);
            };
            f32x4_t z[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 4 * q + e;
                    float sum = acc[i][NB - 1][r];
#pragma unroll
                    for (int b = NB - 2; b >= 0; --b) sum = __builtin_fmaf(sum, 0.00390625f, acc[i][b][r]);
                    z[q][e] = sum;
                }
            if (part) {
#pragma unroll
                for (int q = 0; q < 4; ++q) put(cbase, ldc, col_of(q), z[q]);
                continue;
            }
            if (be.bias != nullptr) {
                if (full) {
                    // the bias of the wave's 32 columns (gated: 16 gates, 16
                    // ups) by scalar loads under one wait, which never waits
                    // for the direct loads in flight (a wait per 8 columns:
                    // 2,325 us instead of 2,258 on the gated 552,960 x 256 ->
                    // 2 x 512).  Tiles of 64 rows load 8 words at a time:
                    // the 32 registers cost their main loop spills (2,048 x
                    // 4096 -> 1024: 165 us instead of 155).
                    const float* b = be.bias + n0 + gw * (EPI == EPI_GATED ? 16 : 32);
                    const float* b1 = EPI == EPI_GATED ? b + p.N : b + 16;
                    const bool upper = (lane >> 5) != 0;
                    auto add = [&](int q, int e, int lo, int hi) __attribute__((always_inline)) {
                        // (opaque copies: otherwise the two selects fold
                        // into an index and a chain of compares)
                        asm("" : "+s"(lo));
                        asm("" : "+s"(hi));
                        z[q][e] = z[q][e] + __int_as_float(upper ? hi : lo);
                    };
                    if constexpr (TH == 128) {
                        i32x16_t bw[2];
                        scalar_load16x2(b, b1, bw[0], bw[1]);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int e = 0; e < 4; ++e) add(q, e, bw[q >> 1][8 * (q & 1) + e], bw[q >> 1][8 * (q & 1) + 4 + e]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const i32x8_t bw = scalar_load8((q >= 2 ? b1 : b) + 8 * (q & 1));
#pragma unroll
                            for (int e = 0; e < 4; ++e) add(q, e, bw[e], bw[4 + e]);
                        }
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        z[q] = z[q] + load4(be.bias + n0 + (EPI == EPI_GATED && q >= 2 ? p.N : 0), col_of(q), cols_left);
                }
            }
            if (has_z) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    put(zbase + (EPI == EPI_GATED && q >= 2 ? p.N : 0), be.ldz, col_of(q), z[q]);
            }
            constexpr int NOUT = EPI == EPI_GATED ? 2 : 4;
            with_act(be.act, [&]<int ACT>() {
#pragma unroll
                for (int q = 0; q < NOUT; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[q][e] = act_value<ACT>(z[q][e]);
            });
#pragma unroll
            for (int q = 0; q < NOUT; ++q) {
                f32x4_t o = z[q];
                if constexpr (EPI == EPI_GATED) o = o * z[q + 2];
                if constexpr (EPI == EPI_ACT)
                    if (has_r) o = o + res[i][q];
                put(cbase, ldc, col_of(q), o);
            }
        }
    };
    const bool unit_alpha = p.alpha == 1.0f;
    auto epilogue_any = [&](const TilePos& w) __attribute__((always_inline)) {
        if constexpr (EPI != EPI_PLAIN)
            block_epilogue(w, reload_epilogue(finish...));
        else if constexpr (SPLIT)
            epilogue.template operator()<true>(w);
        else if (unit_alpha)
            epilogue.template operator()<false>(w);
        else
            epilogue.template operator()<true>(w);
    };

    // Cursors: wm = step of the next M phase, we = the step before it (its
    // tile gets the epilogue when that step was the tile's last), ws = the
    // step after it (split, and its B chunk loaded, in the next U phase),
    // wa = the step of the next A load.
    Walk wm;
    if constexpr (SPLIT) {
        walk_set_item(wm, wc, slot);
    } else {
        wm.seg = 0;
        wm.tn = slot % p.tiles_n;
        wm.m0 = (int64_t)(slot / p.tiles_n) * TH;
        wm.kt = 0;
        wm.kt_end = p.nk;
        wm.item = slot;
        wm.part = 0;
        wm.widx = 0;
        walk_set_tile(wm, wc);
    }
    wm.left = my_items - 1;
    wm.kvalid = wm.kt + 1 < p.nk ? BK : wc.tail_k;
    Walk ws = wm, wa = wm;
    TilePos we{wm.m0, wm.tn, wm.rows, wm.seg, wm.part, wm.widx};
    // Prologue: B chunk of step 0 (each group its half) and group 1's half
    // of B chunk 1, then the FP32 A rows of steps 0 and 1, all issued before
    // one wait that leaves only the step-1 rows in flight (U(0) waits for
    // them); then the split of step 0 into plane buffer 0.  One memory
    // latency before the first MFMA instead of two for group 1: a few us on
    // a GEMM of a few tiles per CU.
    copy_b_half(ws, 0);
    if (grp == 1) {
        Walk w1 = ws;
        walk_next<SPLIT>(w1, wc);
        copy_b_half(w1, 1);
    }
    copy_a32(wa, 0);
    walk_next<SPLIT>(wa, wc);
    copy_a32(wa, 1);
    walk_next<SPLIT>(wa, wc);
    wait_vmcnt<A_ROUNDS>();
    {
        f32x4_t v0[A_ROUNDS];
        load_rows(ws, 0, v0);
        split_rows(v0, 0);
    }
    walk_next<SPLIT>(ws, wc);
    wait_lgkmcnt0();   // the split's LDS writes, published by the barrier
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (grp == 1) __builtin_amdgcn_s_barrier();   // group 1 runs one phase behind group 0

    // The epilogue runs before the U phase's direct loads: its stores then
    // issue ahead of those loads instead of queueing behind them (2-3 %
    // faster than the other order, results identical), and the compiler's
    // waits for its C loads (beta != 0) find no direct load of this phase
    // in flight.  Vector memory operations complete in issue order, so the
    // waits below also cover the stores.
    bool epi = false;       // U(s) runs the epilogue of step s-1's tile
    int bm = 0;             // B buffer of step s: s % 3
    for (int s = 0; s < total; ++s) {
        const int b = s & 1;
        const int bn = bm == 2 ? 0 : bm + 1;   // B buffer of step s+1
        // ---- U(s).  The A rows of step s+1 were loaded in U(s-1) (or the
        // prologue) into staging b^1, after that phase's epilogue stores and
        // half of B chunk s.
        wait_vmcnt<0>();
        f32x4_t sv[A_ROUNDS];
        load_rows(ws, b ^ 1, sv);
        if (epi) {
            epilogue_any(we);
            clear_acc();   // here, not in each epilogue variant: one copy of the clears
        }
        // Group 0 loads its half of B chunk s+1 (ws) into the buffer of step
        // s-2, group 1 its half of chunk s+2 (wa) into that of step s-1;
        // the last readers of each, M(s-2) and M(s-1) of both groups, ended
        // before this phase.  Each group waits for its half at the end of
        // its next M phase, so chunk s+1 is whole before U0(s+1) and both
        // groups read their first B fragments before the U->M barrier.
        if (grp == 0)
            copy_b_half(ws, bn);
        else
            copy_b_half(wa, bn == 2 ? 0 : bn + 1);
        copy_a32(wa, b);   // staging b held step s, split in U(s-1)
        // The first fragments of M(s) are read before the barrier where they
        // are already published: this group's A planes (split in U(s-1),
        // published by the barrier that ended M(s-1)) and B chunk s (both
        // halves landed before the barrier that ended the phase before
        // U0(s)).  They are issued before the split, which gives the
        // staging reads of load_rows longer to land.
        bf16x8_t bfr0[NP], atop0[TM];
        load_afr(b, 0, NP - 1, atop0);
        load_bfr(bm, 0, bfr0);
        split_rows(sv, b ^ 1);   // plane buffer b^1 was last read by M(s-1)
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();   // the split's writes drain during M(s)
        __builtin_amdgcn_sched_barrier(0);
        // ---- M(s) on plane buffer b (split in U(s-1)) and B buffer bm, and
        // the cursor advances for U(s+1).  The MFMAs run in 2 NP groups,
        // (k-half, A plane u) = (0, NP-1) .. (0, 0), (1, NP-1) .. (1, 0); the
        // fragments of each group are read while the group before it issues
        // (the first group's before the barrier above).
        {
            bf16x8_t bq[2][NP], aq[2][TM];
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) bq[0][pl] = bfr0[pl];
#pragma unroll
            for (int i = 0; i < TM; ++i) aq[0][i] = atop0[i];
#pragma unroll
            for (int g = 0; g < 2 * NP; ++g) {
                const int half = g / NP, u = NP - 1 - g % NP;
                if (g + 1 < 2 * NP) {
                    const int nhalf = (g + 1) / NP, nu = NP - 1 - (g + 1) % NP;
                    if (nu == NP - 1) load_bfr(bm, nhalf, bq[nhalf]);
                    load_afr(b, nhalf, nu, aq[(g + 1) & 1]);
                }
                __builtin_amdgcn_sched_barrier(0);
                mfma_u(u, bq[half], aq[g & 1]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        epi = wm.kt == (SPLIT ? wm.kt_end : p.nk) - 1;
        we = TilePos{wm.m0, wm.tn, wm.rows, wm.seg, wm.part, wm.widx};
        // wm, ws, wa are the same sequence one and two steps apart (past the
        // end all stay on the last step): one advance, two copies
        wm = ws;
        ws = wa;
        walk_next<SPLIT>(wa, wc);
        bm = bn;
        // Before the next barrier: this thread's split writes of U(s) are
        // complete (the group reads them in M(s+1)); this group's half of B
        // loaded in U(s) (and the epilogue's stores before it) has landed,
        // while its A load of U(s), issued after it, may still be in flight.
        wait_lgkmcnt0();
        wait_vmcnt<A_ROUNDS>();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    }
    epilogue_any(we);
    wait_vmcnt<0>();   // no direct load may still be writing LDS when the workgroup ends
    if (grp == 0) __builtin_amdgcn_s_barrier();   // matches group 1's extra barrier
}

}  // namespace
}  // namespace emu
