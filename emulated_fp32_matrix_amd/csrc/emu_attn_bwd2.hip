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
#include "emu_attn_device.h"

namespace emu {
namespace {

template <int ND, int W, int NQ, bool SUMS>
__global__ __launch_bounds__(256) void rows_kernel(AttnArgs a, AttnPlan plan, AttnSeconds x, float* delta, float* sums,
                                                   float* go, float* gq)
{
    using T = Team<W>;
    constexpr int LD = Head<ND>::LD, KT = StreamTile<ND, W>::kRows, NK = KT / 16;
    __shared__ __attribute__((aligned(16))) float lds[T::kTeams][4 * KT * LD + 2 * KT];
    float* const tk = lds[T::index()];
    float* const tv = tk + KT * LD;
    float* const tvk = tv + KT * LD;
    float* const tvv = tvk + KT * LD;
    float* const term = tvv + KT * LD;
    float* const vterm = term + KT;
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
    const int64_t all_rows = (int64_t)a.batch * a.queries * a.heads;

    each_piece<W>((int64_t)a.batch * a.kv_heads * plan.own * plan.splits, [&](int64_t piece) {
        const Piece at = piece_of(a, plan, piece);
        const int limit = keys_of(a, at.b);
        int64_t lo, hi;
        range_of(limit, KT, plan.splits, at.split, lo, hi);

        f32x4_t oq[NQ][ND], od[NQ][ND], oa[NQ][ND];
        float top[NQ], over[NQ], del[NQ], mean[NQ], tmean[NQ];   // SUMS: the last two are this range's sums
        const int64_t r0 = (at.own * W + T::wave()) * (16 * NQ) + m;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = r0 + 16 * n;
            const bool valid = r < a.rows;
            const RowAt ra = row_at(a, at.g, valid ? r : 0);
            const int64_t row = row_index(a, at.b, ra);
            load_own(oq[n], row_ptr(x.q, at.b, ra), valid, h, a.dim);
            load_own(od[n], row_ptr(x.dout, at.b, ra), valid, h, a.dim);
            load_own(oa[n], row_ptr(x.vq, at.b, ra), valid && x.vq.data != nullptr, h, a.dim);
            top[n] = x.stats[2 * row];
            over[n] = x.stats[2 * row + 1];
            if constexpr (SUMS) {
                float d = 0.0f;
#pragma unroll
                for (int c = 0; c < ND; ++c) {
                    const f32x4_t o = load4(x.out + row * a.dim, 16 * c + 4 * h, a.dim);
#pragma unroll
                    for (int e = 0; e < 4; ++e) d = __builtin_fmaf(od[n][c][e], o[e], d);
                }
                del[n] = column_sum(d);
                if (valid && h == 0 && at.split == 0) delta[row] = del[n];
                mean[n] = tmean[n] = 0.0f;
            } else {
                del[n] = delta[row];
                mean[n] = tmean[n] = 0.0f;
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

        for (int64_t k0 = lo; k0 < hi; k0 += KT) {
            {
                const auto takes_part = [&](int row) { return key_term(a, at.b, (int)k0 + row, limit) != minus_inf(); };
                const auto rows_of = [&](const emu_heads_t& t) {
                    return [&, t](int row) {
                        return t.data != nullptr && takes_part(row) ? key_ptr(t, at.b, at.g, k0 + row) : nullptr;
                    };
                };
                Tile<ND, KT, T::kThreads> f0, f1;
                f0.fetch(T::thread(), a.dim, rows_of(x.k));
                f1.fetch(T::thread(), a.dim, rows_of(x.v));
                T::sync();
                f0.put(T::thread(), tk);
                f1.put(T::thread(), tv);
                f0.fetch(T::thread(), a.dim, rows_of(x.vk));
                f1.fetch(T::thread(), a.dim, rows_of(x.vv));
                f0.put(T::thread(), tvk);
                f1.put(T::thread(), tvv);
                if (T::thread() < KT) {
                    const int j = (int)k0 + T::thread();
                    const float add = key_term(a, at.b, j, limit);
                    term[T::thread()] = add;
                    vterm[T::thread()] =
                        x.vbias != nullptr && add != minus_inf() ? x.vbias[at.b * x.vbias_b + j * x.vbias_k] : 0.0f;
                }
                T::sync();
            }
#pragma unroll
            for (int t = 0; t < NK; ++t) {
                const int row = 16 * t * LD;
                f32x4_t s[NQ], dp[NQ], gg[NQ], ee[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n) s[n] = dp[n] = gg[n] = ee[n] = f32x4_t{};
                scores<ND, NQ>(tk + row, m, h, oq, s);
                scores<ND, NQ>(tk + row, m, h, oa, gg);
                scores<ND, NQ>(tvk + row, m, h, oq, gg);
                scores<ND, NQ>(tv + row, m, h, od, dp);
                scores<ND, NQ>(tvv + row, m, h, od, ee);
                const f32x4_t add = *reinterpret_cast<const f32x4_t*>(term + 16 * t + 4 * h);
                const f32x4_t vadd = *reinterpret_cast<const f32x4_t*>(vterm + 16 * t + 4 * h);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool dead = add[j] == minus_inf();
                        const float p =
                            dead ? 0.0f : exp_of(__builtin_fmaf(s[n][j], a.scale, add[j]) - top[n]) * over[n];
                        const float g = __builtin_fmaf(gg[n][j], a.scale, vadd[j]);
                        const float d = dp[n][j] - del[n];
                        const float v = __builtin_fmaf(g, d, ee[n][j]);
                        if constexpr (SUMS) {
                            mean[n] = dead ? mean[n] : __builtin_fmaf(p, g, mean[n]);
                            tmean[n] = dead ? tmean[n] : __builtin_fmaf(p, v, tmean[n]);
                        } else {
                            s[n][j] = p;
                            gg[n][j] = dead ? 0.0f : p * (g - mean[n]);
                            dp[n][j] = dead ? 0.0f : p * d;
                            ee[n][j] = dead ? 0.0f : p * (__builtin_fmaf(-mean[n], d + del[n], v) - tmean[n]);
                        }
                    }
                if constexpr (!SUMS) {
                    results<ND, NQ>(tv + row, m, h, gg, ao);    // H v
                    results<ND, NQ>(tvv + row, m, h, s, ao);    // p vv
                    results<ND, NQ>(tk + row, m, h, ee, aq);    // U k
                    results<ND, NQ>(tvk + row, m, h, dp, aq);   // ds vk
                }
            }
        }

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

template <int ND, int W, int NT>
__global__ __launch_bounds__(256) void keys_kernel(AttnArgs a, AttnPlan plan, AttnSeconds x, const float* delta,
                                                   const float* sums, int sum_splits, float* gk, float* gv, float* gb)
{
    using T = Team<W>;
    constexpr int LD = Head<ND>::LD, RT = StreamTile<ND, W>::kRows, NR = RT / 16;
    __shared__ __attribute__((aligned(16))) float lds[T::kTeams][3 * RT * LD + 5 * RT];
    float* const tq = lds[T::index()];
    float* const td = tq + RT * LD;
    float* const ta = td + RT * LD;
    float* const row_stats = ta + RT * LD;   // maxima, 1 / sums, deltas, g, t
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
    const int64_t all_rows = (int64_t)a.batch * a.queries * a.heads;

    each_piece<W>((int64_t)a.batch * a.kv_heads * plan.own * plan.splits, [&](int64_t piece) {
        const Piece at = piece_of(a, plan, piece);
        const int limit = keys_of(a, at.b);
        int64_t lo, hi;
        range_of(a.rows, RT, plan.splits, at.split, lo, hi);

        f32x4_t ok[NT][ND], ov[NT][ND], ovk[NT][ND], ovv[NT][ND], ak[NT][ND], av[NT][ND];
        float add[NT], vadd[NT], bias[NT];
        const int64_t j0 = (at.own * W + T::wave()) * (16 * NT) + m;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t j = j0 + 16 * n;
            add[n] = j < a.keys ? key_term(a, at.b, (int)j, limit) : minus_inf();
            const bool valid = add[n] != minus_inf();
            const int64_t jj = valid ? j : 0;
            load_own(ok[n], key_ptr(x.k, at.b, at.g, jj), valid, h, a.dim);
            load_own(ov[n], key_ptr(x.v, at.b, at.g, jj), valid, h, a.dim);
            load_own(ovk[n], key_ptr(x.vk, at.b, at.g, jj), valid && x.vk.data != nullptr, h, a.dim);
            load_own(ovv[n], key_ptr(x.vv, at.b, at.g, jj), valid && x.vv.data != nullptr, h, a.dim);
            vadd[n] = valid && x.vbias != nullptr ? x.vbias[at.b * x.vbias_b + jj * x.vbias_k] : 0.0f;
            bias[n] = 0.0f;
        }
        clear(ak);
        clear(av);
        // (a team whose keys all take no part has zeros to write)
        if (at.own * W * 16 * NT >= limit) hi = lo;

        for (int64_t r = lo; r < hi; r += RT) {
            {
                const auto rows_of = [&](const emu_heads_t& t) {
                    return [&, t](int row) {
                        return t.data != nullptr && r + row < hi ? row_ptr(t, at.b, row_at(a, at.g, r + row)) : nullptr;
                    };
                };
                Tile<ND, RT, T::kThreads> f0, f1, f2;
                f0.fetch(T::thread(), a.dim, rows_of(x.q));
                f1.fetch(T::thread(), a.dim, rows_of(x.dout));
                f2.fetch(T::thread(), a.dim, rows_of(x.vq));
                T::sync();
                f0.put(T::thread(), tq);
                f1.put(T::thread(), td);
                f2.put(T::thread(), ta);
                if (T::thread() < RT) {
                    const int i = T::thread();
                    const bool valid = r + i < hi;
                    const int64_t row = valid ? row_index(a, at.b, row_at(a, at.g, r + i)) : 0;
                    const float del = valid ? delta[row] : 0.0f;
                    float g = 0.0f, t = 0.0f;
                    for (int s = 0; s < sum_splits && valid; ++s) {
                        g = g + sums[2 * (s * all_rows + row)];
                        t = t + sums[2 * (s * all_rows + row) + 1];
                    }
                    row_stats[i] = valid ? x.stats[2 * row] : 0.0f;
                    row_stats[RT + i] = valid ? x.stats[2 * row + 1] : 0.0f;
                    row_stats[2 * RT + i] = del;
                    row_stats[3 * RT + i] = g;
                    row_stats[4 * RT + i] = __builtin_fmaf(-g, del, t);
                }
                T::sync();
            }
#pragma unroll
            for (int t = 0; t < NR; ++t) {
                const int row = 16 * t * LD, first = 16 * t + 4 * h;
                f32x4_t s[NT], dp[NT], gg[NT], ee[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n] = dp[n] = gg[n] = ee[n] = f32x4_t{};
                scores<ND, NT>(tq + row, m, h, ok, s);
                scores<ND, NT>(ta + row, m, h, ok, gg);
                scores<ND, NT>(tq + row, m, h, ovk, gg);
                scores<ND, NT>(td + row, m, h, ov, dp);
                scores<ND, NT>(td + row, m, h, ovv, ee);
                const f32x4_t top = *reinterpret_cast<const f32x4_t*>(row_stats + first);
                const f32x4_t over = *reinterpret_cast<const f32x4_t*>(row_stats + RT + first);
                const f32x4_t del = *reinterpret_cast<const f32x4_t*>(row_stats + 2 * RT + first);
                const f32x4_t mean = *reinterpret_cast<const f32x4_t*>(row_stats + 3 * RT + first);
                const f32x4_t tmean = *reinterpret_cast<const f32x4_t*>(row_stats + 4 * RT + first);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool dead = add[n] == minus_inf() || r + first + j >= hi;
                        const float p = exp_of(__builtin_fmaf(s[n][j], a.scale, add[n]) - top[j]) * over[j];
                        const float g = __builtin_fmaf(gg[n][j], a.scale, vadd[n]);
                        const float d = dp[n][j] - del[j];
                        const float v = __builtin_fmaf(-mean[j], d + del[j], __builtin_fmaf(g, d, ee[n][j]));
                        gg[n][j] = dead ? 0.0f : p * (g - mean[j]);
                        dp[n][j] = dead ? 0.0f : p * d;
                        ee[n][j] = dead ? 0.0f : p * (v - tmean[j]);
                        bias[n] = bias[n] + ee[n][j];
                    }
                results<ND, NT>(td + row, m, h, gg, av);   // H dout
                results<ND, NT>(tq + row, m, h, ee, ak);   // U q
                results<ND, NT>(ta + row, m, h, dp, ak);   // ds vq
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
            const int64_t to = key_index(a, at.b, at.g, j) + at.split * ((int64_t)a.batch * a.keys * a.kv_heads);
            if (gk != nullptr) store_own(ak[n], a.scale, gk + to * a.dim, h, a.dim);
            if (gv != nullptr) store_own(av[n], 1.0f, gv + to * a.dim, h, a.dim);
            if (gb != nullptr && h == 0)
                gb[(((int64_t)at.b * plan.splits + at.split) * a.kv_heads + at.g) * a.keys + j] = dead ? 0.0f : sum;
        }
    });
}

int64_t pieces(const AttnArgs& a, const AttnPlan& p) { return (int64_t)a.batch * a.kv_heads * p.own * p.splits; }

}  // namespace

hipError_t launch_attn_second_sums(const AttnArgs& a, const AttnPlan& p, const AttnSeconds& x, float* delta,
                                   float* sums, hipStream_t s)
{
    with_shape<1>(a.dim, p, [&]<int ND, int W, int NQ>() {
        rows_kernel<ND, W, NQ, true><<<attn_grid<W>(pieces(a, p)), 256, 0, s>>>(a, p, x, delta, sums, nullptr, nullptr);
    });
    return hipGetLastError();
}

hipError_t launch_attn_second_rows(const AttnArgs& a, const AttnPlan& p, const AttnSeconds& x, const float* delta,
                                   const float* sums, float* gdout, float* gq, float* partial_o, float* partial_q,
                                   hipStream_t s)
{
    const bool cut = p.splits > 1;
    float* const to_o = gdout != nullptr && cut ? partial_o : gdout;
    float* const to_q = gq != nullptr && cut ? partial_q : gq;
    with_shape<1>(a.dim, p, [&]<int ND, int W, int NQ>() {
        rows_kernel<ND, W, NQ, false><<<attn_grid<W>(pieces(a, p)), 256, 0, s>>>(
            a, p, x, const_cast<float*>(delta), const_cast<float*>(sums), to_o, to_q);
    });
    hipError_t e = hipGetLastError();
    const int64_t n = (int64_t)a.batch * a.queries * a.heads * a.dim;
    if (e == hipSuccess && cut && gdout != nullptr) e = launch_attn_join(1, p.splits, n, partial_o, gdout, s);
    if (e == hipSuccess && cut && gq != nullptr) e = launch_attn_join(1, p.splits, n, partial_q, gq, s);
    return e;
}

hipError_t launch_attn_second_keys(const AttnArgs& a, const AttnPlan& p, const AttnSeconds& x, const float* delta,
                                   const float* sums, int sum_splits, float* gk, float* gv, float* gbias,
                                   float* partial_k, float* partial_v, float* partial_b, hipStream_t s)
{
    const bool cut = p.splits > 1, join_bias = gbias != nullptr && (cut || a.kv_heads > 1);
    float* const to_k = gk != nullptr && cut ? partial_k : gk;
    float* const to_v = gv != nullptr && cut ? partial_v : gv;
    float* const to_b = join_bias ? partial_b : gbias;
    with_shape<1>(a.dim, p, [&]<int ND, int W, int NT>() {
        keys_kernel<ND, W, NT><<<attn_grid<W>(pieces(a, p)), 256, 0, s>>>(a, p, x, delta, sums, sum_splits, to_k, to_v, to_b);
    });
    hipError_t e = hipGetLastError();
    const int64_t n = (int64_t)a.batch * a.keys * a.kv_heads * a.dim;
    if (e == hipSuccess && cut && gk != nullptr) e = launch_attn_join(1, p.splits, n, partial_k, gk, s);
    if (e == hipSuccess && cut && gv != nullptr) e = launch_attn_join(1, p.splits, n, partial_v, gv, s);
    if (e == hipSuccess && join_bias)
        e = launch_attn_join(a.batch, (int64_t)p.splits * a.kv_heads, a.keys, partial_b, gbias, s);
    return e;
}

}  // namespace emu
