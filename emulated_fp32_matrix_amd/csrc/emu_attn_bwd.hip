// Attention, backward pass (include/emu_attention.h).
//
// Two passes that make the probabilities again from the forward pass's
// maximum and sum of each row, without atomics: one over the rows (their
// queries and output gradients stay in registers, keys and values stream
// through LDS; it leaves dq, and delta = dout . out for the other), and one
// over the keys (keys and values stay, queries and output gradients stream;
// dk, dv and the bias gradient).  Layouts as in the forward pass.
#include "emu_attn_device.h"

namespace emu {
namespace {

template <int ND, int W, int NQ>
__global__ __launch_bounds__(256) void rows_kernel(AttnArgs a, AttnPlan plan, emu_heads_t dout, emu_heads_t q,
                                                   emu_heads_t k, emu_heads_t v, const float* out, const float* stats,
                                                   float* delta, float* dq, float* partial)
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

        f32x4_t oq[NQ][ND], od[NQ][ND], acc[NQ][ND];
        float top[NQ], over[NQ], del[NQ];
        const int64_t r0 = (at.own * W + T::wave()) * (16 * NQ) + m;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = r0 + 16 * n;
            const bool valid = r < a.rows;
            const RowAt ra = row_at(a, at.g, valid ? r : 0);
            const int64_t row = row_index(a, at.b, ra);
            load_own(oq[n], row_ptr(q, at.b, ra), valid, h, a.dim);
            load_own(od[n], row_ptr(dout, at.b, ra), valid, h, a.dim);
            float d = 0.0f;
#pragma unroll
            for (int c = 0; c < ND; ++c) {
                const f32x4_t o = load4(out + row * a.dim, 16 * c + 4 * h, a.dim);
#pragma unroll
                for (int e = 0; e < 4; ++e) d = __builtin_fmaf(od[n][c][e], o[e], d);
            }
            del[n] = column_sum(d);
            top[n] = stats[2 * row];
            over[n] = stats[2 * row + 1];
            if (valid && h == 0 && at.split == 0) delta[row] = del[n];
        }
        clear(acc);

        for (int64_t k0 = lo; k0 < hi && dq != nullptr; k0 += KT) {
            {
                Tile<ND, KT, T::kThreads> fk, fv;
                const auto takes_part = [&](int row) { return key_term(a, at.b, (int)k0 + row, limit) != minus_inf(); };
                fk.fetch(T::thread(), a.dim, [&](int row) { return takes_part(row) ? key_ptr(k, at.b, at.g, k0 + row) : nullptr; });
                fv.fetch(T::thread(), a.dim, [&](int row) { return takes_part(row) ? key_ptr(v, at.b, at.g, k0 + row) : nullptr; });
                T::sync();
                fk.put(T::thread(), tk);
                fv.put(T::thread(), tv);
                if (T::thread() < KT) term[T::thread()] = key_term(a, at.b, (int)k0 + T::thread(), limit);
                T::sync();
            }
#pragma unroll
            for (int t = 0; t < NK; ++t) {
                f32x4_t s[NQ], dp[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n) s[n] = dp[n] = f32x4_t{};
                scores<ND, NQ>(tk + 16 * t * LD, m, h, oq, s);
                scores<ND, NQ>(tv + 16 * t * LD, m, h, od, dp);
                const f32x4_t add = *reinterpret_cast<const f32x4_t*>(term + 16 * t + 4 * h);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = exp_of(__builtin_fmaf(s[n][j], a.scale, add[j]) - top[n]) * over[n];
                        s[n][j] = add[j] == minus_inf() ? 0.0f : p * (dp[n][j] - del[n]);
                    }
                results<ND, NQ>(tk + 16 * t * LD, m, h, s, acc);
            }
        }

        if (dq == nullptr) return;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = r0 + 16 * n;
            if (r >= a.rows) continue;
            int64_t row = row_index(a, at.b, row_at(a, at.g, r));
            if (plan.splits > 1) row += at.split * ((int64_t)a.batch * a.queries * a.heads);
            store_own(acc[n], a.scale, (plan.splits > 1 ? partial : dq) + row * a.dim, h, a.dim);
        }
    });
}

template <int ND, int W, int NT>
__global__ __launch_bounds__(256) void keys_kernel(AttnArgs a, AttnPlan plan, emu_heads_t dout, emu_heads_t q,
                                                   emu_heads_t k, emu_heads_t v, const float* stats,
                                                   const float* delta, float* dk, float* dv, float* db)
{
    using T = Team<W>;
    constexpr int LD = Head<ND>::LD, RT = StreamTile<ND, W>::kRows, NR = RT / 16;
    __shared__ __attribute__((aligned(16))) float lds[T::kTeams][2 * RT * LD + 3 * RT];
    float* const tq = lds[T::index()];
    float* const td = tq + RT * LD;
    float* const row_stats = td + RT * LD;   // maxima, 1 / sums, deltas
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;

    each_piece<W>((int64_t)a.batch * a.kv_heads * plan.own * plan.splits, [&](int64_t piece) {
        const Piece at = piece_of(a, plan, piece);
        const int limit = keys_of(a, at.b);
        int64_t lo, hi;
        range_of(a.rows, RT, plan.splits, at.split, lo, hi);

        f32x4_t ok[NT][ND], ov[NT][ND], ak[NT][ND], av[NT][ND];
        float add[NT], bias[NT];
        const int64_t j0 = (at.own * W + T::wave()) * (16 * NT) + m;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t j = j0 + 16 * n;
            add[n] = j < a.keys ? key_term(a, at.b, (int)j, limit) : minus_inf();
            const bool valid = add[n] != minus_inf();
            load_own(ok[n], key_ptr(k, at.b, at.g, valid ? j : 0), valid, h, a.dim);
            load_own(ov[n], key_ptr(v, at.b, at.g, valid ? j : 0), valid, h, a.dim);
            bias[n] = 0.0f;
        }
        clear(ak);
        clear(av);
        // (a team whose keys all take no part has zeros to write)
        if (at.own * W * 16 * NT >= limit) hi = lo;

        for (int64_t r = lo; r < hi; r += RT) {
            {
                Tile<ND, RT, T::kThreads> fq, fd;
                fq.fetch(T::thread(), a.dim, [&](int row) {
                    return r + row < hi ? row_ptr(q, at.b, row_at(a, at.g, r + row)) : nullptr;
                });
                fd.fetch(T::thread(), a.dim, [&](int row) {
                    return r + row < hi ? row_ptr(dout, at.b, row_at(a, at.g, r + row)) : nullptr;
                });
                T::sync();
                fq.put(T::thread(), tq);
                fd.put(T::thread(), td);
                if (T::thread() < RT) {
                    const int i = T::thread();
                    const bool valid = r + i < hi;
                    const int64_t row = valid ? row_index(a, at.b, row_at(a, at.g, r + i)) : 0;
                    row_stats[i] = valid ? stats[2 * row] : 0.0f;
                    row_stats[RT + i] = valid ? stats[2 * row + 1] : 0.0f;   // (so that p = 0)
                    row_stats[2 * RT + i] = valid ? delta[row] : 0.0f;
                }
                T::sync();
            }
#pragma unroll
            for (int t = 0; t < NR; ++t) {
                f32x4_t s[NT], dp[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n] = dp[n] = f32x4_t{};
                scores<ND, NT>(tq + 16 * t * LD, m, h, ok, s);
                scores<ND, NT>(td + 16 * t * LD, m, h, ov, dp);
                const f32x4_t top = *reinterpret_cast<const f32x4_t*>(row_stats + 16 * t + 4 * h);
                const f32x4_t over = *reinterpret_cast<const f32x4_t*>(row_stats + RT + 16 * t + 4 * h);
                const f32x4_t del = *reinterpret_cast<const f32x4_t*>(row_stats + 2 * RT + 16 * t + 4 * h);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool dead = add[n] == minus_inf() || r + 16 * t + 4 * h + j >= hi;
                        const float p = exp_of(__builtin_fmaf(s[n][j], a.scale, add[n]) - top[j]) * over[j];
                        s[n][j] = dead ? 0.0f : p;
                        dp[n][j] = dead ? 0.0f : p * (dp[n][j] - del[j]);
                        bias[n] = bias[n] + dp[n][j];
                    }
                results<ND, NT>(td + 16 * t * LD, m, h, s, av);
                results<ND, NT>(tq + 16 * t * LD, m, h, dp, ak);
            }
        }

#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t j = j0 + 16 * n;
            const float sum = column_sum(bias[n]);
            if (j >= a.keys) continue;
            const bool dead = add[n] == minus_inf();
            if (dead) {
#pragma unroll
                for (int t = 0; t < ND; ++t) ak[n][t] = av[n][t] = f32x4_t{};
            }
            int64_t to = key_index(a, at.b, at.g, j);
            to += at.split * ((int64_t)a.batch * a.keys * a.kv_heads);
            if (dk != nullptr) store_own(ak[n], a.scale, dk + to * a.dim, h, a.dim);
            if (dv != nullptr) store_own(av[n], 1.0f, dv + to * a.dim, h, a.dim);
            // (bias partials: [batch][split][key head][key], joined over the middle two)
            if (db != nullptr && h == 0)
                db[(((int64_t)at.b * plan.splits + at.split) * a.kv_heads + at.g) * a.keys + j] = dead ? 0.0f : sum;
        }
    });
}

}  // namespace

hipError_t launch_attn_backward_rows(const AttnArgs& a, const AttnPlan& p, emu_heads_t dout, emu_heads_t q,
                                     emu_heads_t k, emu_heads_t v, const float* out, const float* stats,
                                     float* delta, float* dq, float* partial, hipStream_t s)
{
    with_shape<2>(a.dim, p, [&]<int ND, int W, int NQ>() {
        const int64_t n = (int64_t)a.batch * a.kv_heads * p.own * p.splits;
        rows_kernel<ND, W, NQ><<<attn_grid<W>(n), 256, 0, s>>>(a, p, dout, q, k, v, out, stats, delta, dq, partial);
    });
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.splits > 1 && dq != nullptr)
        e = launch_attn_join(1, p.splits, (int64_t)a.batch * a.queries * a.heads * a.dim, partial, dq, s);
    return e;
}

hipError_t launch_attn_backward_keys(const AttnArgs& a, const AttnPlan& p, emu_heads_t dout, emu_heads_t q,
                                     emu_heads_t k, emu_heads_t v, const float* stats, const float* delta,
                                     float* dk, float* dv, float* dbias, float* partial_k, float* partial_v,
                                     float* partial_b, hipStream_t s)
{
    const bool cut = p.splits > 1, join_bias = dbias != nullptr && (cut || a.kv_heads > 1);
    float* const to_k = dk != nullptr && cut ? partial_k : dk;
    float* const to_v = dv != nullptr && cut ? partial_v : dv;
    float* const to_b = join_bias ? partial_b : dbias;
    with_shape<1>(a.dim, p, [&]<int ND, int W, int NT>() {
        const int64_t n = (int64_t)a.batch * a.kv_heads * p.own * p.splits;
        keys_kernel<ND, W, NT><<<attn_grid<W>(n), 256, 0, s>>>(a, p, dout, q, k, v, stats, delta, to_k, to_v, to_b);
    });
    hipError_t e = hipGetLastError();
    const int64_t n = (int64_t)a.batch * a.keys * a.kv_heads * a.dim;
    if (e == hipSuccess && cut && dk != nullptr) e = launch_attn_join(1, p.splits, n, partial_k, dk, s);
    if (e == hipSuccess && cut && dv != nullptr) e = launch_attn_join(1, p.splits, n, partial_v, dv, s);
    if (e == hipSuccess && join_bias)
        e = launch_attn_join(a.batch, (int64_t)p.splits * a.kv_heads, a.keys, partial_b, dbias, s);
    return e;
}

}  // namespace emu
