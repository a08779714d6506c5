// Internal interface between the C-ABI layer of the attention operators
// (emu_attn_api.hip) and their kernels.  Not installed; callers use
// include/emu_attention.h.
#pragma once

#include <hip/hip_runtime.h>

#include "emu_attention.h"

namespace emu {

// One attention call after validation.  A key and value head's rows are its
// queries times the heads that share it: row r is query r / share, head
// kv_head * share + r % share, so that the sharing heads read keys once.
struct AttnArgs {
    int batch, queries, keys, heads, kv_heads, share, dim;
    int64_t rows;            // queries * share
    uint32_t share_inverse;  // ceil(2^32 / share) where r / share is the upper half of r times it, else 0
    float scale;
    const float* bias;       // key bias or null
    int64_t bias_b, bias_k;
    const uint8_t* mask;     // key mask or null
    int64_t mask_b, mask_k;
    const void* lengths;     // or null
    int lengths_64;
};

// The passes of longer sequences: the forward pass, its backward pass over rows
// and over keys, and that one's (its rows' sums and results share a plan).
enum class AttnPass { forward, rows, keys, second_rows, second_keys };

// Tiles of 16 of its own side that a wave keeps, while two waves fit a SIMD:
// with two, a streamed operand read from LDS serves both. 2 x 16 heads of 2,048
// x 4,096 x 64: forward 437 us with one and 399 with two, by rows 613 and 534;
// 96 wide forward 155 and 138; 32 wide second order by rows 706 and 622 (2 x 16
// heads of 2,000 x 2,048). The passes over keys keep two results, and two tiles
// of them leave no registers to read ahead: 887 us, with one 783; 32 wide the
// same.
constexpr int attn_tiles(AttnPass pass, int dim)
{
    switch (pass) {
    case AttnPass::forward: return dim <= 96 ? 2 : 1;
    case AttnPass::rows: return dim <= 64 ? 2 : 1;
    case AttnPass::second_rows: return dim <= 32 ? 2 : 1;
    default: return 1;
    }
}
// Waves of a SIMD that the registers are divided among: two, though several
// kernels then keep up to 65 registers in memory, except where that costs more
// than the second wave hides. us with one and two: second order over keys of 33
// to 64 wide heads (58 and 61 of them in memory without images, 13 and 14 with)
// 2 x 16 heads of 1,000 x 2,048 x 64 whole call 1,051 and 920, 23 x 8 of 1,331 x 60 x
// 64 513 and 464, 2 x 8 of 2,000 x 50 x 48 113 and 118; the second order's passes of
// 65 to 96 wide ones 2 x 16 of 1,000 x 2,048 x 96 1,523 and 1,552, 8 x 8 of 300 x 60 x
// 80 111 and 127, 8 x 8 of 60 x 300 x 96 132 and 169. Above 96 wide the own side alone
// takes more than half of the registers in the passes that have one here.
constexpr int attn_waves(AttnPass pass, int nd, bool images)
{
    const bool second = pass == AttnPass::second_rows || pass == AttnPass::second_keys;
    if (nd >= 8) return second || pass == AttnPass::keys ? 1 : 2;
    return nd >= 5 && second && (pass == AttnPass::second_keys || !images) ? 1 : 2;
}

// How a pass is cut into pieces of work: a team of `waves` waves (4; 1 in the
// forward pass of few rows) takes `tiles` tiles of 16 (of its own side) per
// wave and one of `splits` ranges of the other side.
// images: the other side is split beforehand (attn_images).
struct AttnPlan {
    int waves, tiles, splits, images;
    int64_t own;             // pieces along the team's own side
    int64_t run;             // neighbouring pieces that go to one XCD
};
AttnPlan attn_plan(const AttnArgs& a, AttnPass pass);

// Tiles of 32 streamed rows of n arrays as they lie in LDS, split into three
// BF16 pieces: [array][piece][row][attn_image_row], in whole KB. Group i of
// eight elements of row r lies at group i ^ attn_image_place(steps of 32 in a
// row, r). LDS has 64 banks of 4 bytes: a row of 256 bytes takes them all, so 16
// rows have group i at 16 places and eight rows their pairs of groups at eight;
// rows of 128 bytes alternate between the banks' halves, which leaves eight
// places and four; rows of 64 (or 192) take their quarters: four and two.
constexpr int kAttnTile = 32;
constexpr int attn_image_row(int dim) { return (dim + 31) / 32 * 32; }
constexpr __host__ __device__ int attn_image_place(int steps, int r)
{
    const int shift = steps % 4 == 0 ? 0 : steps % 2 == 0 ? 1 : 2;   // rows beside each other
    return 2 * ((r & 7) >> shift) + (r >> 3 & 1);
}
constexpr int64_t attn_image_bytes(int dim, int n)
{
    return ((int64_t)n * 3 * kAttnTile * attn_image_row(dim) * 2 + 1023) / 1024 * 1024;
}
// Bytes of all tiles of a side, and the launch that makes them: `n` arrays of
// the keys' shape (keys that take no part: zeros) and `m` of the rows' (either
// may be 0; data null: zeros).
size_t attn_key_images(const AttnArgs& a, int n);
size_t attn_row_images(const AttnArgs& a, int m);
hipError_t launch_attn_images(const AttnArgs& a, int n, const emu_heads_t* keys, void* key_images, int m,
                              const emu_heads_t* rows, void* row_images, hipStream_t s);

// The forward pass; partial: null unless plan.splits > 1.
size_t attn_forward_partial(const AttnArgs& a, const AttnPlan& p);
// images: of k and v, where the plan has them (so below: of the other side's
// arrays, in the order k, v, vk, vv or q, dout, vq).
hipError_t launch_attn_forward(const AttnArgs& a, const AttnPlan& p, emu_heads_t q, emu_heads_t k, emu_heads_t v,
                               const void* images, float* out, float* stats, float* partial, hipStream_t s);

// Its first launch where a team is one wave (at most 16 rows).
hipError_t launch_attn_few(const AttnArgs& a, const AttnPlan& p, emu_heads_t q, emu_heads_t k, emu_heads_t v, float* out,
                           float* stats, float* partial, hipStream_t s);

// Floats of partial sums (0 for one split): of a result with the queries'
// shape, of one with the keys' shape, of the bias gradient.
size_t attn_rows_partial(const AttnArgs& a, const AttnPlan& p);
size_t attn_keys_partial(const AttnArgs& a, const AttnPlan& p);
size_t attn_bias_partial(const AttnArgs& a, const AttnPlan& p);

// out[o][i] = sum over s of in[o][s][i], s in order; outer x inner results.
// Those of a call are one launch; out null, or in itself: nothing to do.
struct AttnJoin {
    int64_t outer, splits, inner;
    const float* in;
    float* out;
};
constexpr int kAttnJoins = 5;
struct AttnJoins {
    int n;
    AttnJoin of[kAttnJoins];
    void add(const AttnJoin& x)
    {
        if (x.out != nullptr && x.in != x.out && x.outer * x.inner > 0) of[n++] = x;
    }
};
hipError_t launch_attn_joins(const AttnJoins& joins, hipStream_t s);

// The passes' results are in place once `joins`, to which they add, has run.
// delta: a float per row, written by the pass over rows and read by the pass
// over keys.  dq may be null (then only delta is written).
hipError_t launch_attn_backward_rows(const AttnArgs& a, const AttnPlan& p, emu_heads_t dout, emu_heads_t q,
                                     emu_heads_t k, emu_heads_t v, const float* out, const float* stats,
                                     const void* images, float* delta, float* dq, float* partial, AttnJoins& joins, hipStream_t s);
hipError_t launch_attn_backward_keys(const AttnArgs& a, const AttnPlan& p, emu_heads_t dout, emu_heads_t q,
                                     emu_heads_t k, emu_heads_t v, const void* images, const float* stats,
                                     const float* delta, float* dk, float* dv, float* dbias, float* partial_k, float* partial_v,
                                     float* partial_b, AttnJoins& joins, hipStream_t s);

// The backward pass's backward pass.
struct AttnSeconds {
    emu_heads_t vq, vk, vv;  // data null: zeros
    const float* vbias;      // or null
    int64_t vbias_b, vbias_k;
    emu_heads_t dout, q, k, v;
    const float* out;
    const float* stats;
};
// sums: [splits][rows of the call][2] partial sums over keys; delta as above.
hipError_t launch_attn_second_sums(const AttnArgs& a, const AttnPlan& p, const AttnSeconds& t, const void* images,
                                   float* delta, float* sums, hipStream_t s);
hipError_t launch_attn_second_rows(const AttnArgs& a, const AttnPlan& p, const AttnSeconds& t, const void* images, const float* delta,
                                   const float* sums, float* gdout, float* gq, float* partial_o, float* partial_q,
                                   AttnJoins& joins, hipStream_t s);
hipError_t launch_attn_second_keys(const AttnArgs& a, const AttnPlan& p, const AttnSeconds& t, const void* images, const float* delta,
                                   const float* sums, int sum_splits, float* gk, float* gv, float* gbias,
                                   float* partial_k, float* partial_v, float* partial_b, AttnJoins& joins, hipStream_t s);

// Short sequences, each direction in one launch: whether a call's are, and
// the launches.  partial: floats of attn_whole_partial().
bool attn_whole(const AttnArgs& a);
inline size_t attn_whole_partial(const AttnArgs& a)
{
    return a.kv_heads > 1 ? (size_t)a.batch * a.keys * a.kv_heads : 0;
}
hipError_t launch_whole_forward(const AttnArgs& a, emu_heads_t q, emu_heads_t k, emu_heads_t v, float* out, float* stats,
                                hipStream_t s);
hipError_t launch_whole_backward(const AttnArgs& a, emu_heads_t dout, emu_heads_t q, emu_heads_t k, emu_heads_t v,
                                 const float* stats, float* dq, float* dk, float* dv, float* dbias, float* partial,
                                 hipStream_t s);
hipError_t launch_whole_second(const AttnArgs& a, const AttnSeconds& x, float* gdout, float* gq, float* gk, float* gv,
                               float* gbias, float* partial, hipStream_t s);

struct RotaryArgs {
    int64_t batch, tokens;
    int heads, dim, pairs, layout, inverse;
    emu_heads_t x;
    const int64_t* positions;
    int64_t pos_b, pos_t;
    const uint64_t* turns;
    float magnitude;
    float* y;
};
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t s);

struct DropoutArgs {
    int64_t rows, cols;
    const float* x;
    int64_t ldx;
    uint64_t threshold;      // of a 32-bit word: 0 .. 2^32
    float scale;
    const int64_t* seed;
    const float* r;          // or null
    int64_t ldr;
    float* y;
    int64_t ldy;
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s);

}  // namespace emu
