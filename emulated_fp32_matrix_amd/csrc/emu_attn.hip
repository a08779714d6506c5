// Attention, forward pass (include/emu_attention.h).
//
// One pass over the keys with the running maximum and sum of the softmax: a
// wave keeps 16 or 32 rows, their queries in registers as the B operand and
// their results as accumulators, both with the row across the lanes, so that
// the softmax's maxima and factors are per lane and a score's registers are
// the next product's operand (emu_attn_device.h).  A team's tile of keys and
// values goes through LDS once for all of its rows.
//
// Few rows are cut along the keys: each range leaves a maximum, a sum and an
// unscaled result, and a second launch joins them in order.
#include "emu_attn_device.h"

namespace emu {
namespace {

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

template <int ND, int W, int NQ>
__global__ __launch_bounds__(256) void forward_kernel(AttnArgs a, AttnPlan plan, emu_heads_t q, emu_heads_t k,
                                                      emu_heads_t v, float* out, float* stats, float* partial)
{
    using T = Team<W>;
    constexpr int LD = Head<ND>::LD, KT = StreamTile<ND, W>::kRows, NK = KT / 16;
    __shared__ __attribute__((aligned(16))) float lds[T::kTeams][2 * KT * LD + KT];
    float* const tk = lds[T::index()];
    float* const tv = tk + KT * LD;
    float* const term = tv + KT * LD;
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;

    each_piece<W>((int64_t)a.batch * a.kv_heads * plan.own * plan.splits, [&](int64_t piece) {
        const Piece at = piece_of(a, plan, piece);
        const int limit = keys_of(a, at.b);
        int64_t lo, hi;
        range_of(limit, KT, plan.splits, at.split, lo, hi);

        f32x4_t own[NQ][ND], acc[NQ][ND];
        float most[NQ], sum[NQ];
        const int64_t r0 = (at.own * W + T::wave()) * (16 * NQ) + m;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = r0 + 16 * n;
            const bool valid = r < a.rows;
            load_own(own[n], row_ptr(q, at.b, row_at(a, at.g, valid ? r : 0)), valid, h, a.dim);
            most[n] = minus_inf();
            sum[n] = 0.0f;
        }
        clear(acc);

        for (int64_t k0 = lo; k0 < hi; k0 += KT) {
            {
                Tile<ND, KT, T::kThreads> fk, fv;
                const auto takes_part = [&](int row) { return key_term(a, at.b, (int)k0 + row, limit) != minus_inf(); };
                fk.fetch(T::thread(), a.dim, [&](int row) { return takes_part(row) ? key_ptr(k, at.b, at.g, k0 + row) : nullptr; });
                fv.fetch(T::thread(), a.dim, [&](int row) { return takes_part(row) ? key_ptr(v, at.b, at.g, k0 + row) : nullptr; });
                T::sync();   // the previous tile has been read
                fk.put(T::thread(), tk);
                fv.put(T::thread(), tv);
                if (T::thread() < KT) term[T::thread()] = key_term(a, at.b, (int)k0 + T::thread(), limit);
                T::sync();
            }
            f32x4_t s[NK][NQ];
#pragma unroll
            for (int t = 0; t < NK; ++t) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) s[t][n] = f32x4_t{};
                scores<ND, NQ>(tk + 16 * t * LD, m, h, own, s[t]);
                const f32x4_t add = *reinterpret_cast<const f32x4_t*>(term + 16 * t + 4 * h);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[t][n][j] = add[j] == minus_inf() ? minus_inf() : __builtin_fmaf(s[t][n][j], a.scale, add[j]);
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float top = s[0][n][0];
#pragma unroll
                for (int t = 0; t < NK; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) top = __builtin_fmaxf(top, s[t][n][j]);
                const float next = __builtin_fmaxf(most[n], column_max(top));
                const float safe = next == minus_inf() ? 0.0f : next;   // (no key so far: all of e^(-inf - 0) = 0)
                const float old = exp_of(most[n] - safe);
                most[n] = next;
                float here = 0.0f;
#pragma unroll
                for (int t = 0; t < NK; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[t][n][j] = exp_of(s[t][n][j] - safe);
                        here = here + s[t][n][j];
                    }
                sum[n] = __builtin_fmaf(sum[n], old, here);
#pragma unroll
                for (int t = 0; t < ND; ++t) acc[n][t] = acc[n][t] * old;
            }
#pragma unroll
            for (int t = 0; t < NK; ++t) results<ND, NQ>(tv + 16 * t * LD, m, h, s[t], acc);
        }

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

// The ranges' results of a row, joined: one wave per row.
__global__ __launch_bounds__(256) void join_forward_kernel(AttnArgs a, AttnPlan plan, float* partial, float* out,
                                                           float* stats)
{
    const int64_t rows = (int64_t)a.batch * a.queries * a.heads;
    const ForwardPartial from = forward_partial(a, plan, partial);
    const int lane = threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.x * 4) {
        float most = minus_inf();
        for (int s = 0; s < plan.splits; ++s) most = __builtin_fmaxf(most, from.ml[2 * (s * rows + row)]);
        const float safe = most == minus_inf() ? 0.0f : most;
        float sum = 0.0f, lo = 0.0f, hi = 0.0f;
        for (int s = 0; s < plan.splits; ++s) {
            const int64_t i = s * rows + row;
            const float f = exp_of(from.ml[2 * i] - safe);
            sum = __builtin_fmaf(from.ml[2 * i + 1], f, sum);
            if (lane < a.dim) lo = __builtin_fmaf(from.o[i * a.dim + lane], f, lo);
            if (lane + 64 < a.dim) hi = __builtin_fmaf(from.o[i * a.dim + lane + 64], f, hi);
        }
        const float over = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (lane < a.dim) out[row * a.dim + lane] = lo * over;
        if (lane + 64 < a.dim) out[row * a.dim + lane + 64] = hi * over;
        if (stats != nullptr && lane == 0) {
            stats[2 * row] = safe;
            stats[2 * row + 1] = over;
        }
    }
}

__global__ __launch_bounds__(256) void join_kernel(int64_t n, int64_t splits, int64_t inner, const float* in, float* out)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t o = i / inner;
        const float* at = in + o * splits * inner + (i - o * inner);
        float sum = at[0];
        for (int64_t s = 1; s < splits; ++s) sum = sum + at[s * inner];
        out[i] = sum;
    }
}

unsigned join_grid(int64_t groups) { return (unsigned)(groups < 65536 ? groups : 65536); }

// Ranges of the other side: enough pieces for 2,048 waves (256 compute units
// of 8), none shorter than `least` of the streamed side.
int splits_for(int64_t waves, int64_t other, int64_t least)
{
    int64_t s = waves > 0 ? 2048 / waves : 1;
    const int64_t most = other / least;
    if (s > most) s = most;
    if (s > 64) s = 64;
    return s < 1 ? 1 : (int)s;
}

// `most`: tiles of 16 per wave that fit its registers.
AttnPlan plan_for(const AttnArgs& a, int64_t own, int64_t other, int most)
{
    AttnPlan p{};
    p.waves = own <= 32 ? 1 : 4;
    p.tiles = most == 1 || own <= 16 || (own > 32 && own <= 64) ? 1 : 2;
    if (p.waves == 1 && own > 16 * p.tiles) p.waves = 4;
    const int64_t each = p.waves * p.tiles * 16;
    p.own = (own + each - 1) / each;
    p.splits = splits_for((int64_t)a.batch * a.kv_heads * p.own * p.waves, other, p.waves == 1 ? 128 : 256);
    return p;
}

}  // namespace

AttnPlan attn_rows_plan(const AttnArgs& a, int order) { return plan_for(a, a.rows, a.keys, a.dim > 64 && order == 2 ? 1 : 2); }
AttnPlan attn_keys_plan(const AttnArgs& a, int) { return plan_for(a, a.keys, a.rows, a.dim > 64 ? 1 : 2); }

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
                               float* out, float* stats, float* partial, hipStream_t s)
{
    with_shape<2>(a.dim, p, [&]<int ND, int W, int NQ>() {
        const int64_t n = (int64_t)a.batch * a.kv_heads * p.own * p.splits;
        forward_kernel<ND, W, NQ><<<attn_grid<W>(n), 256, 0, s>>>(a, p, q, k, v, out, stats, partial);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    join_forward_kernel<<<join_grid(((int64_t)a.batch * a.queries * a.heads + 3) / 4), 256, 0, s>>>(a, p, partial, out, stats);
    return hipGetLastError();
}

hipError_t launch_attn_join(int64_t outer, int64_t splits, int64_t inner, const float* in, float* out, hipStream_t s)
{
    const int64_t n = outer * inner;
    if (n == 0) return hipSuccess;
    join_kernel<<<join_grid((n + 255) / 256), 256, 0, s>>>(n, splits, inner, in, out);
    return hipGetLastError();
}

}  // namespace emu
