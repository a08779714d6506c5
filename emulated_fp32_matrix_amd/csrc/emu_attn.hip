// Attention, forward pass (include/emu_attention.h).
//
// One pass over the keys with the running maximum and sum of the softmax: a
// wave keeps 16 or 32 rows, their queries in registers as the B operand and
// their results as accumulators (emu_attn_device.h), on split operands
// (emu_attn_split.h). A team of four waves shares a tile of keys and values in
// LDS, split once for all of its rows.
//
// Where there are few pieces of work, or sequences of different lengths, they
// are cut along the keys: each range leaves a maximum, a sum and an unscaled
// result, and a second launch joins them in order.
//
// Bound by the matrix units at the power limit: 2 x 16 heads of 2,048 x 4,096 x
// 64, 68.7 GFLOP, in 327 to 410 us by the clock that the power leaves (168 to
// 210 TFLOP/s; FP32 library product 153), the matrix units busy half of the
// time and the vector units, for the softmax and the splits of its weights, the
// other half.
#include "emu_attn_split.h"

namespace emu {
namespace {

constexpr int kMostSplits = 64;

// How far a row's running maximum may lag behind before sums and results are
// rescaled: most tiles then leave them as they are. Weights reach e^kSlack, and
// their exponents' rounding grows with kSlack (exp_of(): 0.9 2^-24 of the weight
// at 1, 3.7 at 4). us with 0, 1, 2 and 4: 4 x 8 heads of 2,000 x 2,000 x 32 122.5,
// 120.8, 119.9, 119.4; 2 x 16 of 2,048 x 4,096 x 64 365, 363, 362, 362; 8 x 8 of 250
// x 1,000 x 64 48.4, 47.8, 47.8, 47.6.
constexpr float kSlack = 1.0f;

template <int ND, int NQ, bool IMAGES>
__global__ __launch_bounds__(64 * kTeam, attn_waves(AttnPass::forward, ND, IMAGES)) void forward_kernel(AttnArgs a, AttnPlan plan, emu_heads_t q, emu_heads_t k,
                                                         emu_heads_t v, const char* images, float* out, float* stats,
                                                         float* partial)
{
    using T = Team<kTeam>;
    using S = Stream<ND, 2, 1, true, IMAGES, attn_waves(AttnPass::forward, ND, IMAGES)>;
    __shared__ __attribute__((aligned(16))) char lds[S::kBuffers * S::kBytes];
    S stream{lds};
    stream.clear();
    stagger();
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;

    T::each_piece(pieces_of(a, plan), plan.run, [&](int64_t piece) {
        const Piece at = piece_of(a, plan, piece);
        const int limit = keys_of(a, at.b);
        int64_t lo, hi;
        range_of(limit, kStreamRows, plan.splits, at.split, lo, hi);

        Split8 own[NQ][Heads<ND>::KS];
        f32x4_t acc[NQ][ND];
        float most[NQ], sum[NQ];
        const int64_t r0 = (at.own * kTeam + T::wave()) * (16 * NQ) + m;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = r0 + 16 * n;
            const bool valid = r < a.rows;
            load_own<ND>(own[n], row_ptr(q, at.b, row_at(a, at.g, valid ? r : 0)), valid, h, a.dim);
            most[n] = minus_inf();
            sum[n] = 0.0f;
        }
        clear(acc);

        const auto number = [&](int64_t first, float* to) { to[0] = key_term(a, at.b, (int)first + T::thread(), limit); };
        stream.run_keys(a, at, images, lo, hi, number, [&](int64_t, const uint16_t* arrays, const float* numbers) {
            const Terms term(numbers, h);
            f32x4_t s[2][NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[0][n] = s[1][n] = f32x4_t{};
            scores<ND, S::kPiece, true, NQ>(arrays, m, h, own, s);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[t][n][j] = __builtin_fmaf(s[t][n][j], a.scale, term.of[t][j]);
            // The factor's exponent follows the maximum only where that has
            // grown by more than kSlack since.
            bool grown = false;
            float next[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float top = s[0][n][0];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) top = __builtin_fmaxf(top, s[t][n][j]);
                next[n] = column_max(top);
                grown = grown || next[n] > most[n] + kSlack;
            }
            if (__any(grown)) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    next[n] = __builtin_fmaxf(most[n], next[n]);
                    const float old = most[n] == next[n] ? 1.0f : exp_of(most[n] - next[n]);
                    most[n] = next[n];
                    sum[n] = sum[n] * old;
#pragma unroll
                    for (int t = 0; t < ND; ++t) acc[n][t] = acc[n][t] * old;
                }
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const float safe = most[n] == minus_inf() ? 0.0f : most[n];   // (no key so far: all of e^(-inf - 0) = 0)
                float here = 0.0f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[t][n][j] = exp_of(s[t][n][j] - safe);
                        here = here + s[t][n][j];
                    }
                sum[n] = sum[n] + here;
            }
            results<ND, S::kPiece, true, NQ>(arrays + S::kArray, m, h, s, acc);
        }, k, v);

#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = r0 + 16 * n;
            const float total = column_sum(sum[n]);
            if (r >= a.rows) continue;
            const int64_t row = row_index(a, at.b, row_at(a, at.g, r));
            if (plan.splits > 1) {
                const ForwardPartial to = forward_partial(a, plan, partial);
                const int64_t i = at.split * ((int64_t)a.batch * a.queries * a.heads) + row;
                store_own(acc[n], 1.0f, to.o + i * a.dim, h, a.dim);
                if (h == 0) {
                    to.ml[2 * i] = most[n];
                    to.ml[2 * i + 1] = total;
                }
            } else {
                const float over = total == 0.0f ? 0.0f : 1.0f / total;
                store_own(acc[n], over, out + row * a.dim, h, a.dim);
                if (stats != nullptr && h == 0) {
                    stats[2 * row] = most[n] == minus_inf() ? 0.0f : most[n];
                    stats[2 * row + 1] = over;
                }
            }
        }
    });
}

// The ranges' results of a row, joined in order: a workgroup per row, whose
// groups of COLS / 4 threads have every GROUPS-th range, four columns a thread,
// all of them requested at once: 4 us for
// 128 rows of 64 ranges of 64, with a column a thread in turn 8.
template <int COLS>
__global__ __launch_bounds__(256) void join_many_kernel(AttnArgs a, AttnPlan plan, float* partial, float* out, float* stats)
{
    constexpr int QUADS = COLS / 4, GROUPS = 256 / QUADS, EACH = kMostSplits / GROUPS;
    __shared__ __attribute__((aligned(16))) float parts[4][COLS];
    static_assert(kMostSplits == 64, "a lane per range");
    const int64_t rows = (int64_t)a.batch * a.queries * a.heads;
    const ForwardPartial from = forward_partial(a, plan, partial);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = threadIdx.x % QUADS * 4, group = threadIdx.x / QUADS;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        f32x4_t x[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int s = i * GROUPS + group;
            x[i] = s < plan.splits ? load4(from.o + (s * rows + row) * a.dim, col, a.dim) : f32x4_t{};
        }
        const bool there = lane < plan.splits;
        const float2 ml = there ? *reinterpret_cast<const float2*>(from.ml + 2 * (lane * rows + row)) : float2{minus_inf(), 0.0f};
        float most = ml.x;
#pragma unroll
        for (int i = 1; i < 64; i *= 2) most = __builtin_fmaxf(most, __shfl_xor(most, i, 64));
        const float safe = most == minus_inf() ? 0.0f : most;
        const float f = there ? exp_of(ml.x - safe) : 0.0f;
        const float sum = lane_sum<64>(ml.y * f);
        const float over = sum == 0.0f ? 0.0f : 1.0f / sum;
        f32x4_t acc = {};
#pragma unroll
        for (int i = 0; i < EACH; ++i) acc = acc + x[i] * __shfl(f, i * GROUPS + group, 64);
#pragma unroll
        for (int i = QUADS; i < 64; i *= 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = acc[e] + __shfl_xor(acc[e], i, 64);
        __syncthreads();   // the previous row's have been read
        if (lane < QUADS) *reinterpret_cast<f32x4_t*>(&parts[wave][col]) = acc;
        __syncthreads();
        if ((int)threadIdx.x < a.dim) {
            const float all = (parts[0][threadIdx.x] + parts[1][threadIdx.x]) + (parts[2][threadIdx.x] + parts[3][threadIdx.x]);
            out[row * a.dim + threadIdx.x] = all * over;
        }
        if (stats != nullptr && threadIdx.x == 0) {
            stats[2 * row] = safe;
            stats[2 * row + 1] = over;
        }
    }
}

// The same of up to kFewSplits ranges: a thread per four columns.
constexpr int kFewSplits = 8;

__global__ __launch_bounds__(256) void join_few_kernel(AttnArgs a, AttnPlan plan, float* partial, float* out, float* stats)
{
    const int64_t rows = (int64_t)a.batch * a.queries * a.heads;
    const ForwardPartial from = forward_partial(a, plan, partial);
    const int quads = (a.dim + 3) / 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * quads; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / quads;
        const int col = (int)(i - row * quads) * 4;
        float most = minus_inf(), m[kFewSplits];
#pragma unroll
        for (int s = 0; s < kFewSplits; ++s) {
            m[s] = s < plan.splits ? from.ml[2 * (s * rows + row)] : minus_inf();
            most = __builtin_fmaxf(most, m[s]);
        }
        const float safe = most == minus_inf() ? 0.0f : most;
        float sum = 0.0f;
        f32x4_t acc = {};
#pragma unroll
        for (int s = 0; s < kFewSplits; ++s) {
            if (s >= plan.splits) continue;
            const float f = exp_of(m[s] - safe);
            sum = __builtin_fmaf(from.ml[2 * (s * rows + row) + 1], f, sum);
            acc = acc + load4(from.o + (s * rows + row) * a.dim, col, a.dim) * f;
        }
        const float over = sum == 0.0f ? 0.0f : 1.0f / sum;
        store4(out + row * a.dim, col, a.dim, acc * over);
        if (stats != nullptr && col == 0) {
            stats[2 * row] = safe;
            stats[2 * row + 1] = over;
        }
    }
}

// blockIdx.y: which of the sums.
__global__ __launch_bounds__(256) void join_kernel(AttnJoins j)
{
    AttnJoin x = j.of[0];   // (chosen, not indexed: arguments stay in scalar registers)
#pragma unroll
    for (int i = 1; i < kAttnJoins; ++i)
        if (blockIdx.y == i) x = j.of[i];
    const int64_t n = x.outer * x.inner;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t o = x.outer == 1 ? 0 : i / x.inner;
        const float* at = x.in + o * x.splits * x.inner + (i - o * x.inner);
        float sum = at[0];
        for (int64_t s = 1; s < x.splits; ++s) sum = sum + at[s * x.inner];
        x.out[i] = sum;
    }
}

unsigned join_grid(int64_t groups) { return (unsigned)(groups < 65536 ? groups : 65536); }

// Teams that stream the same side, from which on it is split beforehand. The
// splitting itself costs a launch and the bytes, and each team saves a fifth of
// its time: 8 x 8 heads of 250 x 1,000 x 64 (two teams) forward 44 us without, 35
// + 17 with, by rows 60 and 47 + 11; 2 x 16 of 2,048 x 4,096 x 64 (16 teams)
// forward 497 and 399 + 32, by keys 970 and 759 + 12.
constexpr int image_teams(AttnPass pass) { return pass == AttnPass::forward ? 4 : 2; }

// Ranges of the other side for a wave each of few rows: as many as make 2,048
// waves (256 compute units of 8), none shorter than 128 keys.
int few_splits(int64_t waves, int64_t other)
{
    int64_t s = 2048 / waves;
    if (s > other / 128) s = other / 128;
    return s < 1 ? 1 : s > kMostSplits ? kMostSplits : (int)s;
}

// Ranges of the other side for teams: the number with the least time, in tiles
// of the streamed side. The compute units have `resident` teams each at once;
// such a round takes a range and about 6 tiles' time to begin and end a piece,
// a last one with a compute unit per team 0.8 of it (0.67 to 0.88 measured).
// The join takes 2 tiles' time and 0.003 a piece. Of sequences that differ in
// length (`ragged`) the long ones end last, by half a range on average. (Of the
// passes over rows: those over keys are counted with the teams of all keys, also
// of those past their sequence's length, which leave at once; the host does not
// know the lengths.)
// Measured against at least 256 of the other side a range and 2,048 waves: 3 x
// 8 heads of 333 x 515 x 40, forward 27 -> 23 us, second order by rows 89 -> 71;
// 7 x 6 of 257 x 777 x 80 ragged, second order by keys 143 -> 137; 21 x 8 of 200
// x 1,918 x 48 ragged, second order by rows 657 -> 614.
int splits_for(int64_t teams, int64_t other, int resident, bool ragged)
{
    constexpr int kUnits = 256;
    const int64_t tiles = (other + kStreamRows - 1) / kStreamRows, slots = kUnits * resident;
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= kMostSplits && (s == 1 || s <= tiles); ++s) {
        const int64_t n = teams * s, rest = n % slots, range = (tiles + s - 1) / s;
        const double rounds = (double)(n / slots) + (rest == 0 ? 0.0 : rest <= kUnits && resident > 1 ? 0.8 : 1.0);
        const double time = rounds * (double)(range + 6) + (ragged ? 0.5 * (double)range : 0.0) + (s > 1 ? 2.0 + 0.003 * (double)n : 0.0);
        if (s == 1 || time < least) {
            best = s;
            least = time;
        }
        if (n > 8 * slots) break;   // (the join alone costs more from here)
    }
    return best;
}

}  // namespace

AttnPlan attn_plan(const AttnArgs& a, AttnPass pass)
{
    const bool keys = pass == AttnPass::keys || pass == AttnPass::second_keys;
    const int64_t own = keys ? a.keys : a.rows, other = keys ? a.rows : a.keys;
    AttnPlan p{};
    // The forward pass has a kernel of its own for few rows: 16 rows of 8 x 8
    // heads over 2,048 keys of 64 in 21 us, with tiles of 64 rows 31; a query's
    // four heads over up to 8,192 keys 22 and 47.
    p.waves = pass == AttnPass::forward && own <= 16 ? 1 : 4;
    p.tiles = own <= 64 ? 1 : attn_tiles(pass, a.dim);
    const int64_t each = p.waves * p.tiles * 16;
    p.own = (own + each - 1) / each;
    p.images = p.waves == 4 && p.own >= image_teams(pass);
    const int64_t pieces = (int64_t)a.batch * a.kv_heads * p.own;
    const int nd = a.dim > 96 ? 8 : (a.dim + 15) / 16;   // as with_shape()
    p.splits = pieces == 0      ? 1
               : p.waves == 1 ? few_splits(pieces, other)
                              : splits_for(pieces, other, attn_waves(pass, nd, p.images), !keys && a.lengths != nullptr);
    // a key head's pieces, if there are 16 such runs for each XCD; a wave's few
    // rows share their keys with no other piece
    const int64_t head = p.own * p.splits, even = pieces * p.splits / 128;
    p.run = p.waves == 1 ? 1 : head < even ? head : even < 1 ? 1 : even;
    return p;
}

size_t attn_forward_partial(const AttnArgs& a, const AttnPlan& p)
{
    return p.splits > 1 ? (size_t)p.splits * a.batch * a.queries * a.heads * (a.dim + 2) : 0;
}
size_t attn_rows_partial(const AttnArgs& a, const AttnPlan& p)
{
    return p.splits > 1 ? (size_t)p.splits * a.batch * a.queries * a.heads * a.dim : 0;
}
size_t attn_keys_partial(const AttnArgs& a, const AttnPlan& p)
{
    return p.splits > 1 ? (size_t)p.splits * a.batch * a.keys * a.kv_heads * a.dim : 0;
}
size_t attn_bias_partial(const AttnArgs& a, const AttnPlan& p)
{
    return p.splits > 1 || a.kv_heads > 1 ? (size_t)p.splits * a.batch * a.keys * a.kv_heads : 0;
}

hipError_t launch_attn_forward(const AttnArgs& a, const AttnPlan& p, emu_heads_t q, emu_heads_t k, emu_heads_t v,
                               const void* images, float* out, float* stats, float* partial, hipStream_t s)
{
    hipError_t e = hipSuccess;
    if (p.waves == 1) {
        e = launch_attn_few(a, p, q, k, v, out, stats, partial, s);
    } else {
        with_shape<AttnPass::forward>(a.dim, p, [&]<int ND, int NQ, bool IMAGES>() {
            forward_kernel<ND, NQ, IMAGES><<<Team<kTeam>::grid(pieces_of(a, p), p.run), 64 * kTeam, 0, s>>>(
                a, p, q, k, v, static_cast<const char*>(images), out, stats, partial);
        });
        e = hipGetLastError();
    }
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t rows = (int64_t)a.batch * a.queries * a.heads;
    const unsigned grid = join_grid(rows);
    if (p.splits <= kFewSplits)
        join_few_kernel<<<join_grid((rows * ((a.dim + 3) / 4) + 255) / 256), 256, 0, s>>>(a, p, partial, out, stats);
    else if (a.dim <= 32)
        join_many_kernel<32><<<grid, 256, 0, s>>>(a, p, partial, out, stats);
    else if (a.dim <= 64)
        join_many_kernel<64><<<grid, 256, 0, s>>>(a, p, partial, out, stats);
    else
        join_many_kernel<128><<<grid, 256, 0, s>>>(a, p, partial, out, stats);
    return hipGetLastError();
}

hipError_t launch_attn_joins(const AttnJoins& joins, hipStream_t s)
{
    if (joins.n == 0) return hipSuccess;
    int64_t most = 0;
    for (int i = 0; i < joins.n; ++i) {
        const int64_t n = joins.of[i].outer * joins.of[i].inner;
        if (n > most) most = n;
    }
    join_kernel<<<dim3(join_grid((most + 255) / 256), joins.n), 256, 0, s>>>(joins);
    return hipGetLastError();
}

}  // namespace emu
