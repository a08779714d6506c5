// Attention of few rows over many keys, forward pass
// (include/emu_attention.h): single queries against an encoder's states.
//
// Bound by the keys' and values' bytes. A wave has up to 16 rows (a query's
// heads that share a key head among them) and a range of the keys, which it
// reads straight into the operands of its products: no LDS, and the next 16
// keys are requested before the present ones are used, so that a compute
// unit's waves keep 64 KB and more on their way. The ranges' results are joined
// by a second launch (emu_attn.hip). Eight sequences of up to 8,192 keys, 4 key
// heads of 64 (67.6 MB read, 2.2 written) in 20 to 22 us: 3.2 to 3.5 TB/s, since all
// sequences are cut into the same number of ranges and the longest one's waves go
// on alone; and the join 4 to 5.
#include "emu_attn_f32.h"

namespace emu {
namespace {

using T = Team<1, 4>;

// 16 keys and values: rows m of the scores, and rows 4 h + j of the results'
// transposed operand.
template <int ND, bool WHOLE>
struct Keys {
    static constexpr int VT = Head<ND>::VT, NC = Head<ND>::NC;
    typedef float vec_t __attribute__((ext_vector_type(VT), aligned(4)));
    f32x4_t k[ND];
    float v[4][ND];
    float term;   // of key m

    __device__ __forceinline__ void load(const AttnArgs& a, const Piece& at, const emu_heads_t& kk, const emu_heads_t& vv, int64_t first,
                                         int limit, int m, int h)
    {
        term = key_term(a, at.b, (int)first + m, limit);
        const int64_t last = limit - 1;
        const float* const row = key_ptr(kk, at.b, at.g, first + m < last ? first + m : last);
#pragma unroll
        for (int c = 0; c < ND; ++c)
            k[c] = WHOLE ? *reinterpret_cast<const f32x4u_t*>(row + 16 * c + 4 * h) : load4(row, 16 * c + 4 * h, a.dim);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t key = first + 4 * h + j;
            const float* const from = key_ptr(vv, at.b, at.g, key < last ? key : last);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = 16 * VT * c + VT * m;
                if constexpr (VT == 1) {
                    v[j][c] = WHOLE || d < a.dim ? from[d] : 0.0f;
                } else if (WHOLE || d + VT <= a.dim) {
                    const vec_t x = *reinterpret_cast<const vec_t*>(from + d);
#pragma unroll
                    for (int u = 0; u < VT; ++u) v[j][VT * c + u] = x[u];
                } else {
#pragma unroll
                    for (int u = 0; u < VT; ++u) v[j][VT * c + u] = d + u < a.dim ? from[d + u] : 0.0f;
                }
            }
        }
    }
};

template <int ND, bool WHOLE>
__global__ __launch_bounds__(256, ND <= 4 ? 2 : 1) void few_kernel(AttnArgs a, AttnPlan plan, emu_heads_t q, emu_heads_t k,
                                                                   emu_heads_t v, float* out, float* stats, float* partial)
{
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
    T::each_piece(pieces_of(a, plan), plan.run, [&](int64_t piece) {
        const Piece at = piece_of(a, plan, piece);
        const int limit = keys_of(a, at.b);
        int64_t lo, hi;
        range_of(limit, kAttnTile, plan.splits, at.split, lo, hi);
        const int64_t r = at.own * 16 + m;
        const bool valid = r < a.rows;
        f32x4_t own[ND], acc[1][ND];
        load_own(own, row_ptr(q, at.b, row_at(a, at.g, valid ? r : 0)), valid, h, a.dim);
        clear_own(acc);
        float most = minus_inf(), sum = 0.0f;
        const auto add = [&](Keys<ND, WHOLE>& x) {
            if (__any(x.term == minus_inf())) {
                if (__all(x.term == minus_inf())) return;   // nothing to add, whatever the rows hold
                // what keys that take no part hold is dropped
#pragma unroll
                for (int c = 0; c < ND; ++c) x.k[c] = x.term == minus_inf() ? f32x4_t{} : x.k[c];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool dead = __shfl(x.term, 4 * h + j, 64) == minus_inf();
#pragma unroll
                    for (int t = 0; t < ND; ++t) x.v[j][t] = dead ? 0.0f : x.v[j][t];
                }
            }
            f32x4_t s = {}, s2 = {};   // (two chains)
#pragma unroll
            for (int c = 0; c < ND; ++c)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    s = mfma4(x.k[c][e], own[c][e], s);
                    s2 = mfma4(x.k[c][e + 1], own[c][e + 1], s2);
                }
            float top = minus_inf();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = __builtin_fmaf(s[j] + s2[j], a.scale, __shfl(x.term, 4 * h + j, 64));
                top = __builtin_fmaxf(top, s[j]);
            }
            const float next = __builtin_fmaxf(most, column_max(top));
            const float safe = next == minus_inf() ? 0.0f : next;
            const float old = exp_of(most - safe);
            most = next;
            float here = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = exp_of(s[j] - safe);
                here = here + s[j];
            }
            sum = __builtin_fmaf(sum, old, here);
#pragma unroll
            for (int t = 0; t < ND; ++t) acc[0][t] = acc[0][t] * old;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int t = 0; t < ND; ++t) acc[0][t] = mfma4(x.v[j][t], s[j], acc[0][t]);
        };
        Keys<ND, WHOLE> even, odd;
        if (lo < hi) even.load(a, at, k, v, lo, limit, m, h);
        for (int64_t first = lo; first < hi; first += 32) {
            const bool more = first + 16 < hi, again = first + 32 < hi;
            if (more) odd.load(a, at, k, v, first + 16, limit, m, h);
            add(even);
            if (again) even.load(a, at, k, v, first + 32, limit, m, h);
            if (more) add(odd);
        }
        const float total = column_sum(sum);
        if (!valid) return;
        const int64_t row = row_index(a, at.b, row_at(a, at.g, r));
        if (plan.splits > 1) {
            const ForwardPartial to = forward_partial(a, plan, partial);
            const int64_t i = at.split * ((int64_t)a.batch * a.queries * a.heads) + row;
            store_own(acc[0], 1.0f, to.o + i * a.dim, h, a.dim);
            if (h == 0) {
                to.ml[2 * i] = most;
                to.ml[2 * i + 1] = total;
            }
            return;
        }
        const float over = total == 0.0f ? 0.0f : 1.0f / total;
        store_own(acc[0], over, out + row * a.dim, h, a.dim);
        if (stats != nullptr && h == 0) {
            stats[2 * row] = most == minus_inf() ? 0.0f : most;
            stats[2 * row + 1] = over;
        }
    });
}

}  // namespace

hipError_t launch_attn_few(const AttnArgs& a, const AttnPlan& p, emu_heads_t q, emu_heads_t k, emu_heads_t v, float* out,
                           float* stats, float* partial, hipStream_t s)
{
    const unsigned grid = T::grid(pieces_of(a, p), p.run);
    const auto run = [&]<int ND>() {
        if (a.dim == 16 * ND)
            few_kernel<ND, true><<<grid, 256, 0, s>>>(a, p, q, k, v, out, stats, partial);
        else
            few_kernel<ND, false><<<grid, 256, 0, s>>>(a, p, q, k, v, out, stats, partial);
    };
    if (a.dim <= 16)
        run.template operator()<1>();
    else if (a.dim <= 32)
        run.template operator()<2>();
    else if (a.dim <= 48)
        run.template operator()<3>();
    else if (a.dim <= 64)
        run.template operator()<4>();
    else if (a.dim <= 80)
        run.template operator()<5>();
    else if (a.dim <= 96)
        run.template operator()<6>();
    else
        run.template operator()<8>();
    return hipGetLastError();
}

}  // namespace emu
