// Attention, the backward pass of its backward pass
// (include/emu_attention.h), for training on forces.
//
// With G = scale (vq K^T + Q vk^T) + vbias, E = dout vv^T and dp = dout V^T per
// row, everything follows from p and two sums of each row, g = sum p G and t =
// sum p T.  Three passes that make the probabilities again: the rows' sums
// first (T's own sum needs g only as a factor: t = sum p (G (dp - delta) + E) -
// g delta), then the results over the rows and over the keys as in the
// backward pass.  Taking the sums first keeps the differences G - g and T - t
// whole before they are multiplied; one pass with running results would take
// them between sums.
// It costs products: a step of training on forces runs 31 where 19 have to be made
// (the sums' five again, and the scores in every pass).
//
// Bound by the matrix units with few waves beside them, since the own side's
// pieces and results fill the registers: 2 x 16 heads of 1,000 x 2,048 x 64, 8.4
// GFLOP a product, in 255 us for the sums (5 products, 164 TFLOP/s), 407 by rows
// (9, 186) and 369 by keys (8, 182).
#include "emu_attn_split.h"

namespace emu {
namespace {

template <int ND, int NQ, bool IMAGES, bool SUMS>
__global__ __launch_bounds__(64 * kTeam, attn_waves(AttnPass::second_rows, ND, IMAGES)) void rows_kernel(AttnArgs a, AttnPlan plan, AttnSeconds x, const char* images, float* delta, float* sums,
                                                      float* go, float* gq)
{
    using T = Team<kTeam>;
    using S = Stream<ND, 4, 2, true, IMAGES, attn_waves(AttnPass::second_rows, ND, IMAGES)>;
    constexpr bool AHEAD = ND <= 4 || attn_waves(AttnPass::second_rows, ND, IMAGES) == 1;
    constexpr int KS = Heads<ND>::KS;
    __shared__ __attribute__((aligned(16))) char lds[S::kBuffers * S::kBytes];
    S stream{lds};
    stream.clear();
    stagger();
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
    const int64_t all_rows = (int64_t)a.batch * a.queries * a.heads;

    T::each_piece(pieces_of(a, plan), plan.run, [&](int64_t piece) {
        const Piece at = piece_of(a, plan, piece);
        const int limit = keys_of(a, at.b);
        int64_t lo, hi;
        range_of(limit, kStreamRows, plan.splits, at.split, lo, hi);

        Split8 oq[NQ][KS], od[NQ][KS], oa[NQ][KS];
        float top[NQ], over[NQ], del[NQ], mean[NQ], tmean[NQ];   // SUMS: the last two are this range's sums
        const int64_t r0 = (at.own * kTeam + T::wave()) * (16 * NQ) + m;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = r0 + 16 * n;
            const bool valid = r < a.rows;
            const RowAt ra = row_at(a, at.g, valid ? r : 0);
            const int64_t row = row_index(a, at.b, ra);
            load_own<ND>(oq[n], row_ptr(x.q, at.b, ra), valid, h, a.dim);
            load_own<ND>(od[n], row_ptr(x.dout, at.b, ra), valid, h, a.dim);
            load_own<ND>(oa[n], row_ptr(x.vq, at.b, ra), valid && x.vq.data != nullptr, h, a.dim);
            top[n] = x.stats[2 * row];
            over[n] = x.stats[2 * row + 1];
            mean[n] = tmean[n] = 0.0f;
            if constexpr (SUMS) {
                del[n] = row_dot<ND>(row_ptr(x.dout, at.b, ra), x.out + row * a.dim, h, a.dim);
                if (valid && h == 0 && at.split == 0) delta[row] = del[n];
            } else {
                del[n] = delta[row];
                for (int s = 0; s < plan.splits; ++s) {
                    mean[n] = mean[n] + sums[2 * (s * all_rows + row)];
                    tmean[n] = tmean[n] + sums[2 * (s * all_rows + row) + 1];
                }
                tmean[n] = __builtin_fmaf(-mean[n], del[n], tmean[n]);
            }
        }
        f32x4_t ao[SUMS ? 1 : NQ][ND], aq[SUMS ? 1 : NQ][ND];
        clear(ao);
        clear(aq);

        const auto number = [&](int64_t first, float* to) {
            to[0] = key_term(a, at.b, (int)first + T::thread(), limit);
            to[1] = x.vbias != nullptr && to[0] != minus_inf() ? x.vbias[at.b * x.vbias_b + (first + T::thread()) * x.vbias_k]
                                                               : 0.0f;
        };
        stream.run_keys(a, at, images, lo, hi, number, [&](int64_t, const uint16_t* arrays, const float* numbers) {
            const Terms term(numbers, h);
            const uint16_t *const tk = arrays, *const tv = tk + S::kArray, *const tvk = tv + S::kArray,
                           *const tvv = tvk + S::kArray;
            f32x4_t s[2][NQ], dp[2][NQ], gg[2][NQ], ee[2][NQ];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int n = 0; n < NQ; ++n) s[t][n] = dp[t][n] = gg[t][n] = ee[t][n] = f32x4_t{};
            scores<ND, S::kPiece, AHEAD, NQ>(tk, m, h, oq, s);
            scores<ND, S::kPiece, AHEAD, NQ>(tk, m, h, oa, gg);
            scores<ND, S::kPiece, AHEAD, NQ>(tvk, m, h, oq, gg);
            scores<ND, S::kPiece, AHEAD, NQ>(tv, m, h, od, dp);
            scores<ND, S::kPiece, AHEAD, NQ>(tvv, m, h, od, ee);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f32x4_t vadd = *reinterpret_cast<const f32x4_t*>(numbers + kStreamRows + 16 * t + 4 * h);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = exp_of(__builtin_fmaf(s[t][n][j], a.scale, term.of[t][j]) - top[n]) * over[n];
                        const float g = __builtin_fmaf(gg[t][n][j], a.scale, vadd[j]);
                        const float d = dp[t][n][j] - del[n];
                        const float v = __builtin_fmaf(g, d, ee[t][n][j]);
                        if constexpr (SUMS) {
                            mean[n] = __builtin_fmaf(p, g, mean[n]);
                            tmean[n] = __builtin_fmaf(p, v, tmean[n]);
                        } else {
                            s[t][n][j] = p;
                            gg[t][n][j] = p * (g - mean[n]);
                            ee[t][n][j] = p * (__builtin_fmaf(-mean[n], dp[t][n][j], v) - tmean[n]);
                            dp[t][n][j] = p * d;
                        }
                    }
            }
            if constexpr (!SUMS) {
                results<ND, S::kPiece, AHEAD, NQ>(tv, m, h, gg, ao);    // H v
                results<ND, S::kPiece, AHEAD, NQ>(tvv, m, h, s, ao);    // p vv
                results<ND, S::kPiece, AHEAD, NQ>(tk, m, h, ee, aq);    // U k
                results<ND, S::kPiece, AHEAD, NQ>(tvk, m, h, dp, aq);   // ds vk
            }
        }, x.k, x.v, x.vk, x.vv);

#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = r0 + 16 * n;
            if constexpr (SUMS) {
                const float g = column_sum(mean[n]), t = column_sum(tmean[n]);
                if (r < a.rows && h == 0) {
                    const int64_t i = at.split * all_rows + row_index(a, at.b, row_at(a, at.g, r));
                    sums[2 * i] = g;
                    sums[2 * i + 1] = t;
                }
            } else {
                if (r >= a.rows) continue;
                const int64_t i = at.split * all_rows + row_index(a, at.b, row_at(a, at.g, r));
                if (go != nullptr) store_own(ao[n], 1.0f, go + i * a.dim, h, a.dim);
                if (gq != nullptr) store_own(aq[n], a.scale, gq + i * a.dim, h, a.dim);
            }
        }
    });
}

template <int ND, int NT, bool IMAGES>
__global__ __launch_bounds__(64 * kTeam, attn_waves(AttnPass::second_keys, ND, IMAGES)) void keys_kernel(AttnArgs a, AttnPlan plan, AttnSeconds x, const char* images, const float* delta,
                                                      const float* sums, int sum_splits, float* gk, float* gv, float* gb)
{
    using T = Team<kTeam>;
    using S = Stream<ND, 3, 5, false, IMAGES, attn_waves(AttnPass::second_keys, ND, IMAGES)>;
    constexpr bool AHEAD = attn_waves(AttnPass::second_keys, ND, IMAGES) == 1;
    constexpr int KS = Heads<ND>::KS;
    __shared__ __attribute__((aligned(16))) char lds[S::kBuffers * S::kBytes];
    S stream{lds};
    stream.clear();
    stagger();
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
    const int64_t all_rows = (int64_t)a.batch * a.queries * a.heads;

    T::each_piece(pieces_of(a, plan), plan.run, [&](int64_t piece) {
        const Piece at = piece_of(a, plan, piece);
        const int limit = keys_of(a, at.b);
        int64_t lo, hi;
        range_of(a.rows, kStreamRows, plan.splits, at.split, lo, hi);

        Split8 ok[NT][KS], ov[NT][KS], ovk[NT][KS], ovv[NT][KS];
        f32x4_t ak[NT][ND], av[NT][ND];
        float add[NT], vadd[NT], bias[NT];
        const int64_t j0 = (at.own * kTeam + T::wave()) * (16 * NT) + m;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t j = j0 + 16 * n;
            add[n] = j < a.keys ? key_term(a, at.b, (int)j, limit) : minus_inf();
            const bool valid = add[n] != minus_inf();
            const int64_t jj = valid ? j : 0;
            load_own<ND>(ok[n], key_ptr(x.k, at.b, at.g, jj), valid, h, a.dim);
            load_own<ND>(ov[n], key_ptr(x.v, at.b, at.g, jj), valid, h, a.dim);
            load_own<ND>(ovk[n], key_ptr(x.vk, at.b, at.g, jj), valid && x.vk.data != nullptr, h, a.dim);
            load_own<ND>(ovv[n], key_ptr(x.vv, at.b, at.g, jj), valid && x.vv.data != nullptr, h, a.dim);
            vadd[n] = valid && x.vbias != nullptr ? x.vbias[at.b * x.vbias_b + jj * x.vbias_k] : 0.0f;
            bias[n] = 0.0f;
        }
        clear(ak);
        clear(av);
        // (a team whose keys all take no part has zeros to write)
        if (at.own * kTeam * 16 * NT >= limit) hi = lo;

        // maxima, 1 / sums, deltas, g, t; behind the last row p = e^-inf 0
        const auto number = [&](int64_t first, float* to) {
            const bool valid = first + T::thread() < hi;
            const int64_t row = valid ? row_index(a, at.b, row_at(a, at.g, first + T::thread())) : 0;
            float g = 0.0f, t = 0.0f;
            for (int s = 0; s < sum_splits && valid; ++s) {
                g = g + sums[2 * (s * all_rows + row)];
                t = t + sums[2 * (s * all_rows + row) + 1];
            }
            to[0] = valid ? x.stats[2 * row] : __builtin_inff();
            to[1] = valid ? x.stats[2 * row + 1] : 0.0f;
            to[2] = valid ? delta[row] : 0.0f;
            to[3] = g;
            to[4] = __builtin_fmaf(-g, to[2], t);
        };
        stream.run_rows(a, at, images, lo, hi, number, [&](int64_t, const uint16_t* arrays, const float* numbers) {
            const uint16_t *const tq = arrays, *const td = tq + S::kArray, *const ta = td + S::kArray;
            f32x4_t s[2][NT], dp[2][NT], gg[2][NT], ee[2][NT];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n) s[t][n] = dp[t][n] = gg[t][n] = ee[t][n] = f32x4_t{};
            scores<ND, S::kPiece, AHEAD, NT>(tq, m, h, ok, s);
            scores<ND, S::kPiece, AHEAD, NT>(ta, m, h, ok, gg);
            scores<ND, S::kPiece, AHEAD, NT>(tq, m, h, ovk, gg);
            scores<ND, S::kPiece, AHEAD, NT>(td, m, h, ov, dp);
            scores<ND, S::kPiece, AHEAD, NT>(td, m, h, ovv, ee);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float* const nums = numbers + 16 * t + 4 * h;
                const f32x4_t top = *reinterpret_cast<const f32x4_t*>(nums);
                const f32x4_t over = *reinterpret_cast<const f32x4_t*>(nums + kStreamRows);
                const f32x4_t del = *reinterpret_cast<const f32x4_t*>(nums + 2 * kStreamRows);
                const f32x4_t mean = *reinterpret_cast<const f32x4_t*>(nums + 3 * kStreamRows);
                const f32x4_t tmean = *reinterpret_cast<const f32x4_t*>(nums + 4 * kStreamRows);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // (a key that takes no part has e^-inf; what NaN in a row leaves there is dropped at the end)
                        const float p = exp_of(__builtin_fmaf(s[t][n][j], a.scale, add[n]) - top[j]) * over[j];
                        const float g = __builtin_fmaf(gg[t][n][j], a.scale, vadd[n]);
                        const float d = dp[t][n][j] - del[j];
                        const float v = __builtin_fmaf(-mean[j], dp[t][n][j], __builtin_fmaf(g, d, ee[t][n][j]));
                        gg[t][n][j] = p * (g - mean[j]);
                        dp[t][n][j] = p * d;
                        ee[t][n][j] = p * (v - tmean[j]);
                        bias[n] = bias[n] + ee[t][n][j];
                    }
            }
            results<ND, S::kPiece, AHEAD, NT>(td, m, h, gg, av);   // H dout
            results<ND, S::kPiece, AHEAD, NT>(tq, m, h, ee, ak);   // U q
            results<ND, S::kPiece, AHEAD, NT>(ta, m, h, dp, ak);   // ds vq
        }, x.q, x.dout, x.vq);

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
            if (gk != nullptr) store_own(ak[n], a.scale, gk + to * a.dim, h, a.dim);
            if (gv != nullptr) store_own(av[n], 1.0f, gv + to * a.dim, h, a.dim);
            if (gb != nullptr && h == 0)
                gb[(((int64_t)at.b * plan.splits + at.split) * a.kv_heads + at.g) * a.keys + j] = dead ? 0.0f : sum;
        }
    });
}

}  // namespace

hipError_t launch_attn_second_sums(const AttnArgs& a, const AttnPlan& p, const AttnSeconds& x, const void* images,
                                   float* delta, float* sums, hipStream_t s)
{
    with_shape<AttnPass::second_rows>(a.dim, p, [&]<int ND, int NQ, bool IMAGES>() {
        rows_kernel<ND, NQ, IMAGES, true><<<Team<kTeam>::grid(pieces_of(a, p), p.run), 64 * kTeam, 0, s>>>(a, p, x, static_cast<const char*>(images), delta, sums, nullptr, nullptr);
    });
    return hipGetLastError();
}

hipError_t launch_attn_second_rows(const AttnArgs& a, const AttnPlan& p, const AttnSeconds& x, const void* images, const float* delta,
                                   const float* sums, float* gdout, float* gq, float* partial_o, float* partial_q,
                                   AttnJoins& joins, hipStream_t s)
{
    const bool cut = p.splits > 1;
    float* const to_o = gdout != nullptr && cut ? partial_o : gdout;
    float* const to_q = gq != nullptr && cut ? partial_q : gq;
    with_shape<AttnPass::second_rows>(a.dim, p, [&]<int ND, int NQ, bool IMAGES>() {
        rows_kernel<ND, NQ, IMAGES, false><<<Team<kTeam>::grid(pieces_of(a, p), p.run), 64 * kTeam, 0, s>>>(
            a, p, x, static_cast<const char*>(images), const_cast<float*>(delta), const_cast<float*>(sums), to_o, to_q);
    });
    const int64_t n = (int64_t)a.batch * a.queries * a.heads * a.dim;
    joins.add({1, p.splits, n, to_o, gdout});
    joins.add({1, p.splits, n, to_q, gq});
    return hipGetLastError();
}

hipError_t launch_attn_second_keys(const AttnArgs& a, const AttnPlan& p, const AttnSeconds& x, const void* images, const float* delta,
                                   const float* sums, int sum_splits, float* gk, float* gv, float* gbias,
                                   float* partial_k, float* partial_v, float* partial_b, AttnJoins& joins, hipStream_t s)
{
    const bool cut = p.splits > 1, join_bias = gbias != nullptr && (cut || a.kv_heads > 1);
    float* const to_k = gk != nullptr && cut ? partial_k : gk;
    float* const to_v = gv != nullptr && cut ? partial_v : gv;
    float* const to_b = join_bias ? partial_b : gbias;
    with_shape<AttnPass::second_keys>(a.dim, p, [&]<int ND, int NT, bool IMAGES>() {
        keys_kernel<ND, NT, IMAGES><<<Team<kTeam>::grid(pieces_of(a, p), p.run), 64 * kTeam, 0, s>>>(a, p, x, static_cast<const char*>(images), delta, sums, sum_splits, to_k, to_v, to_b);
    });
    const int64_t n = (int64_t)a.batch * a.keys * a.kv_heads * a.dim;
    joins.add({1, p.splits, n, to_k, gk});
    joins.add({1, p.splits, n, to_v, gv});
    joins.add({a.batch, (int64_t)p.splits * a.kv_heads, a.keys, to_b, gbias});
    return hipGetLastError();
}

}  // namespace emu
