// Attention, backward pass (include/emu_attention.h).
//
// Two passes that make the probabilities again from the forward pass's
// maximum and sum of each row, without atomics: one over the rows (their
// queries and output gradients stay in registers, keys and values stream
// through LDS; it leaves dq, and delta = dout . out for the other), and one
// over the keys (keys and values stay, queries and output gradients stream;
// dk, dv and the bias gradient).  Layouts as in the forward pass.
//
// Bound as the forward pass is: 2 x 16 heads of 2,048 x 4,096 x 64 in 437 to 540
// us by rows (3 products, 103 GFLOP: 191 to 236 TFLOP/s) and 639 to 760 by keys
// (4 products, 137 GFLOP: 181 to 215).
#include "emu_attn_split.h"

namespace emu {
namespace {

template <int ND, int NQ, bool IMAGES>
__global__ __launch_bounds__(64 * kTeam, attn_waves(AttnPass::rows, ND, IMAGES)) void rows_kernel(AttnArgs a, AttnPlan plan, emu_heads_t dout, emu_heads_t q,
                                                      emu_heads_t k, emu_heads_t v, const char* images, const float* out,
                                                      const float* stats, float* delta, float* dq, float* partial)
{
    using T = Team<kTeam>;
    using S = Stream<ND, 2, 1, true, IMAGES, attn_waves(AttnPass::rows, ND, IMAGES)>;
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

        Split8 oq[NQ][Heads<ND>::KS], od[NQ][Heads<ND>::KS];
        f32x4_t acc[NQ][ND];
        float top[NQ], over[NQ], del[NQ];
        const int64_t r0 = (at.own * kTeam + T::wave()) * (16 * NQ) + m;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = r0 + 16 * n;
            const bool valid = r < a.rows;
            const RowAt ra = row_at(a, at.g, valid ? r : 0);
            const int64_t row = row_index(a, at.b, ra);
            load_own<ND>(oq[n], row_ptr(q, at.b, ra), valid, h, a.dim);
            load_own<ND>(od[n], row_ptr(dout, at.b, ra), valid, h, a.dim);
            del[n] = row_dot<ND>(row_ptr(dout, at.b, ra), out + row * a.dim, h, a.dim);
            top[n] = stats[2 * row];
            over[n] = stats[2 * row + 1];
            if (valid && h == 0 && at.split == 0) delta[row] = del[n];
        }
        clear(acc);

        const auto number = [&](int64_t first, float* to) { to[0] = key_term(a, at.b, (int)first + T::thread(), limit); };
        stream.run_keys(a, at, images, lo, dq != nullptr ? hi : lo, number,
                        [&](int64_t, const uint16_t* arrays, const float* numbers) {
            const Terms term(numbers, h);
            f32x4_t s[2][NQ], dp[2][NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[0][n] = s[1][n] = dp[0][n] = dp[1][n] = f32x4_t{};
            scores<ND, S::kPiece, true, NQ>(arrays, m, h, oq, s);
            scores<ND, S::kPiece, true, NQ>(arrays + S::kArray, m, h, od, dp);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = exp_of(__builtin_fmaf(s[t][n][j], a.scale, term.of[t][j]) - top[n]) * over[n];
                        s[t][n][j] = p * (dp[t][n][j] - del[n]);
                    }
            results<ND, S::kPiece, true, NQ>(arrays, m, h, s, acc);
        }, k, v);

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

template <int ND, int NT, bool IMAGES>
__global__ __launch_bounds__(64 * kTeam, attn_waves(AttnPass::keys, ND, IMAGES)) void keys_kernel(AttnArgs a, AttnPlan plan, emu_heads_t dout, emu_heads_t q,
                                                      emu_heads_t k, emu_heads_t v, const char* images,
                                                      const float* stats, const float* delta, float* dk, float* dv, float* db)
{
    using T = Team<kTeam>;
    using S = Stream<ND, 2, 3, false, IMAGES, attn_waves(AttnPass::keys, ND, IMAGES)>;
    __shared__ __attribute__((aligned(16))) char lds[S::kBuffers * S::kBytes];
    S stream{lds};
    stream.clear();
    stagger();
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;

    T::each_piece(pieces_of(a, plan), plan.run, [&](int64_t piece) {
        const Piece at = piece_of(a, plan, piece);
        const int limit = keys_of(a, at.b);
        int64_t lo, hi;
        range_of(a.rows, kStreamRows, plan.splits, at.split, lo, hi);

        Split8 ok[NT][Heads<ND>::KS], ov[NT][Heads<ND>::KS];
        f32x4_t ak[NT][ND], av[NT][ND];
        float add[NT], bias[NT];
        const int64_t j0 = (at.own * kTeam + T::wave()) * (16 * NT) + m;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t j = j0 + 16 * n;
            add[n] = j < a.keys ? key_term(a, at.b, (int)j, limit) : minus_inf();
            const bool valid = add[n] != minus_inf();
            load_own<ND>(ok[n], key_ptr(k, at.b, at.g, valid ? j : 0), valid, h, a.dim);
            load_own<ND>(ov[n], key_ptr(v, at.b, at.g, valid ? j : 0), valid, h, a.dim);
            bias[n] = 0.0f;
        }
        clear(ak);
        clear(av);
        // (a team whose keys all take no part has zeros to write)
        if (at.own * kTeam * 16 * NT >= limit) hi = lo;

        // maxima, 1 / sums, deltas; behind the last row p = e^-inf 0
        const auto number = [&](int64_t first, float* to) {
            const bool valid = first + T::thread() < hi;
            const int64_t row = valid ? row_index(a, at.b, row_at(a, at.g, first + T::thread())) : 0;
            to[0] = valid ? stats[2 * row] : __builtin_inff();
            to[1] = valid ? stats[2 * row + 1] : 0.0f;
            to[2] = valid ? delta[row] : 0.0f;
        };
        stream.run_rows(a, at, images, lo, hi, number, [&](int64_t, const uint16_t* arrays, const float* numbers) {
            f32x4_t s[2][NT], dp[2][NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[0][n] = s[1][n] = dp[0][n] = dp[1][n] = f32x4_t{};
            scores<ND, S::kPiece, true, NT>(arrays, m, h, ok, s);
            scores<ND, S::kPiece, true, NT>(arrays + S::kArray, m, h, ov, dp);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float* const row = numbers + 16 * t + 4 * h;
                const f32x4_t top = *reinterpret_cast<const f32x4_t*>(row);
                const f32x4_t over = *reinterpret_cast<const f32x4_t*>(row + kStreamRows);
                const f32x4_t del = *reinterpret_cast<const f32x4_t*>(row + 2 * kStreamRows);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // (a key that takes no part has e^-inf; what NaN in a row leaves there is dropped at the end)
                        s[t][n][j] = exp_of(__builtin_fmaf(s[t][n][j], a.scale, add[n]) - top[j]) * over[j];
                        dp[t][n][j] = s[t][n][j] * (dp[t][n][j] - del[j]);
                        bias[n] = bias[n] + dp[t][n][j];
                    }
            }
            results<ND, S::kPiece, true, NT>(arrays + S::kArray, m, h, s, av);
            results<ND, S::kPiece, true, NT>(arrays, m, h, dp, ak);
        }, q, dout);

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
            const int64_t to = key_index(a, at.b, at.g, j) + at.split * ((int64_t)a.batch * a.keys * a.kv_heads);
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
                                     const void* images, float* delta, float* dq, float* partial, AttnJoins& joins, hipStream_t s)
{
    with_shape<AttnPass::rows>(a.dim, p, [&]<int ND, int NQ, bool IMAGES>() {
        rows_kernel<ND, NQ, IMAGES><<<Team<kTeam>::grid(pieces_of(a, p), p.run), 64 * kTeam, 0, s>>>(a, p, dout, q, k, v, static_cast<const char*>(images), out, stats, delta, dq, partial);
    });
    if (p.splits > 1) joins.add({1, p.splits, (int64_t)a.batch * a.queries * a.heads * a.dim, partial, dq});
    return hipGetLastError();
}

hipError_t launch_attn_backward_keys(const AttnArgs& a, const AttnPlan& p, emu_heads_t dout, emu_heads_t q,
                                     emu_heads_t k, emu_heads_t v, const void* images, const float* stats,
                                     const float* delta, float* dk, float* dv, float* dbias, float* partial_k, float* partial_v,
                                     float* partial_b, AttnJoins& joins, hipStream_t s)
{
    const bool cut = p.splits > 1, join_bias = dbias != nullptr && (cut || a.kv_heads > 1);
    float* const to_k = dk != nullptr && cut ? partial_k : dk;
    float* const to_v = dv != nullptr && cut ? partial_v : dv;
    float* const to_b = join_bias ? partial_b : dbias;
    with_shape<AttnPass::keys>(a.dim, p, [&]<int ND, int NT, bool IMAGES>() {
        keys_kernel<ND, NT, IMAGES><<<Team<kTeam>::grid(pieces_of(a, p), p.run), 64 * kTeam, 0, s>>>(a, p, dout, q, k, v, static_cast<const char*>(images), stats, delta, to_k, to_v, to_b);
    });
    const int64_t n = (int64_t)a.batch * a.keys * a.kv_heads * a.dim;
    joins.add({1, p.splits, n, to_k, dk});
    joins.add({1, p.splits, n, to_v, dv});
    joins.add({a.batch, (int64_t)p.splits * a.kv_heads, a.keys, to_b, dbias});
    return hipGetLastError();
}

}  // namespace emu
