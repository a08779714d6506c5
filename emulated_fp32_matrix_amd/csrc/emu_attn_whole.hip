// Attention of short sequences (include/emu_attention.h): the tokens around
// an atom, up to 48 rows and keys.
//
// One wave has a sequence and key head whole: its probabilities stay in
// registers from the first product to the last, so that each direction is one
// launch that reads and writes every array once, keeps no delta, and makes
// the probabilities once instead of once per pass. A tensor's rows are loaded
// straight into the operands of the scores; where the results need them
// transposed, they go through a few KB of the wave's own LDS. Gradients of
// the keys need the weights with the keys across the lanes: those are
// transposed through the same LDS, which costs less than making them again.
//
// Bound by memory: 17,280 x 8 heads of 32 x 32 x 32, a tenth of their keys out of
// reach and not read, forward (2.16 GB) in 442 us, 4.9 TB/s; backward (3.92 GB) in
// 835, 4.7; second order (6.19 GB) in 1,680, 3.7, where 12 products (709 us at
// FP32's rate) lie beside the memory (1,283) only in part. Of three tiles a SIMD has
// one wave: forward above 48 wide, backward above 32, in the second order at every
// width (there 56, 138 and 210 registers of 32, 48 and 64 wide heads are in memory).
#include "emu_attn_f32.h"

namespace emu {
namespace {

using T = Team<1, 4>;

// (neighbouring heads lie beside each other in memory)
__host__ __device__ __forceinline__ int64_t whole_run(const AttnArgs& a) { return ((int64_t)a.batch * a.kv_heads + 31) / 32; }

template <int ND, int NT>
struct Whole {
    static constexpr int LD = Head<ND>::LD, LM = 16 * NT + 4;
    static constexpr int kFloats = 16 * NT * (LD > LM ? LD : LM);   // a wave's LDS
    typedef f32x4_t Frag[NT][ND];
    typedef f32x4_t Mat[NT][NT];   // [streamed tile][own tile], as scores() leaves it

    int m, h;
    float* lds;

    // x[t][n] += (tile t of a) . (tile n of b)
    __device__ __forceinline__ void scores(const Frag& a, const Frag& b, Mat& x) const
    {
#pragma unroll
        for (int c = 0; c < ND; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n) x[t][n] = mfma4(a[t][c][s], b[n][c][s], x[t][n]);
    }

    // acc[n] += a^T . w[.][n], a through LDS
    __device__ __forceinline__ void results(const Frag& a, const Mat& w, Frag& acc) const
    {
        T::sync();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < ND; ++c)
                *reinterpret_cast<f32x4_t*>(lds + (16 * t + m) * LD + 16 * c + 4 * h) = a[t][c];
        T::sync();
#pragma unroll
        for (int t = 0; t < NT; ++t) results_of<ND, NT>(lds + 16 * t * LD, m, h, w[t], acc);
    }

    // x with streamed and own sides exchanged
    __device__ __forceinline__ void exchange(Mat& x) const
    {
        T::sync();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<f32x4_t*>(lds + (16 * n + m) * LM + 16 * t + 4 * h) = x[t][n];
        T::sync();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][t][j] = lds[(16 * n + 4 * h + j) * LM + 16 * t + m];
    }

    static __device__ __forceinline__ void clear(Mat& x)
    {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n) x[t][n] = f32x4_t{};
    }
};

// The wave's sequence and head, its keys' terms and the loads and stores of
// its rows.
template <int ND, int NT>
struct Problem {
    const AttnArgs& a;
    int b, g, m, h, limit;
    float term[NT][4];        // of key 16 t + 4 h + j: as the scores have them
    float term_m[NT];         // of key 16 t + m: as the loads have them

    __device__ __forceinline__ Problem(const AttnArgs& args, int64_t piece, int m_, int h_) : a(args), m(m_), h(h_)
    {
        b = (int)(piece / a.kv_heads);
        g = (int)(piece - (int64_t)b * a.kv_heads);
        limit = keys_of(a, b);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            term_m[t] = key_term(a, b, 16 * t + m, limit);
#pragma unroll
            for (int j = 0; j < 4; ++j) term[t][j] = __shfl(term_m[t], 4 * h + j, 64);
        }
    }
    __device__ __forceinline__ bool dead(int t, int j) const { return term[t][j] == minus_inf(); }
    __device__ __forceinline__ bool has_row(int n) const { return 16 * n + m < a.rows; }
    __device__ __forceinline__ RowAt row(int n) const { return row_at(a, g, has_row(n) ? 16 * n + m : 0); }

    __device__ __forceinline__ void load_rows(f32x4_t (&f)[NT][ND], const emu_heads_t& x) const
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) load_own(f[n], row_ptr(x, b, row(n)), has_row(n) && x.data != nullptr, h, a.dim);
    }
    __device__ __forceinline__ void load_keys(f32x4_t (&f)[NT][ND], const emu_heads_t& x) const
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const bool valid = term_m[t] != minus_inf() && x.data != nullptr;
            load_own(f[t], key_ptr(x, b, g, valid ? 16 * t + m : 0), valid, h, a.dim);
        }
    }
    __device__ __forceinline__ void store_rows(const f32x4_t (&f)[NT][ND], float scale, float* to) const
    {
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (has_row(n)) store_own(f[n], scale, to + row_index(a, b, row(n)) * a.dim, h, a.dim);
    }
    __device__ __forceinline__ void store_keys(f32x4_t (&f)[NT][ND], float scale, float* to) const
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (16 * t + m >= a.keys) continue;
            if (term_m[t] == minus_inf()) {
#pragma unroll
                for (int c = 0; c < ND; ++c) f[t][c] = f32x4_t{};
            }
            store_own(f[t], scale, to + key_index(a, b, g, 16 * t + m) * a.dim, h, a.dim);
        }
    }
    // sums over the rows of w, which has the keys across the lanes
    __device__ __forceinline__ void store_bias(const f32x4_t (&w)[NT][NT], float* to) const
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float sum = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = sum + w[n][t][j];
            sum = column_sum(sum);
            if (h == 0 && 16 * t + m < a.keys)
                to[((int64_t)b * a.kv_heads + g) * a.keys + 16 * t + m] = term_m[t] == minus_inf() ? 0.0f : sum;
        }
    }
    // scores to probabilities by the forward pass's statistics
    __device__ __forceinline__ void probabilities(f32x4_t (&s)[NT][NT], const float* stats) const
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t r = row_index(a, b, row(n));
            const float top = stats[2 * r], over = has_row(n) ? stats[2 * r + 1] : 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[t][n][j] = dead(t, j) || !has_row(n)
                                     ? 0.0f
                                     : exp_of(__builtin_fmaf(s[t][n][j], a.scale, term[t][j]) - top) * over;
        }
    }
};

template <int ND, int NT>
__global__ __launch_bounds__(256) void forward_kernel(AttnArgs a, emu_heads_t q, emu_heads_t k, emu_heads_t v, float* out,
                                                      float* stats)
{
    using W = Whole<ND, NT>;
    __shared__ __attribute__((aligned(16))) float lds[4][W::kFloats];
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
    const W w{m, h, lds[T::index()]};
    T::each_piece((int64_t)a.batch * a.kv_heads, whole_run(a), [&](int64_t piece) {
        const Problem<ND, NT> p(a, piece, m, h);
        typename W::Frag fq, fk, fv, acc;
        typename W::Mat s;
        p.load_keys(fk, k);
        p.load_rows(fq, q);
        p.load_keys(fv, v);
        W::clear(s);
        w.scores(fk, fq, s);
        float over[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float top = minus_inf();
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[t][n][j] = p.dead(t, j) ? minus_inf() : __builtin_fmaf(s[t][n][j], a.scale, p.term[t][j]);
                    top = __builtin_fmaxf(top, s[t][n][j]);
                }
            top = column_max(top);
            top = top == minus_inf() ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[t][n][j] = exp_of(s[t][n][j] - top);
                    sum = sum + s[t][n][j];
                }
            sum = column_sum(sum);
            over[n] = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (stats != nullptr && h == 0 && p.has_row(n)) {
                const int64_t r = row_index(a, p.b, p.row(n));
                stats[2 * r] = top;
                stats[2 * r + 1] = over[n];
            }
        }
        clear_own(acc);
        w.results(fv, s, acc);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (p.has_row(n)) store_own(acc[n], over[n], out + row_index(a, p.b, p.row(n)) * a.dim, h, a.dim);
    });
}

template <int ND, int NT>
__global__ __launch_bounds__(256, NT < 3 && ND * NT <= 4 ? 3 : ND * NT <= 8 ? 2 : 1) void backward_kernel(AttnArgs a, emu_heads_t dout, emu_heads_t q, emu_heads_t k,
                                                       emu_heads_t v, const float* stats, float* dq, float* dk,
                                                       float* dv, float* db)
{
    using W = Whole<ND, NT>;
    __shared__ __attribute__((aligned(16))) float lds[4][W::kFloats];
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
    const W w{m, h, lds[T::index()]};
    T::each_piece((int64_t)a.batch * a.kv_heads, whole_run(a), [&](int64_t piece) {
        const Problem<ND, NT> p(a, piece, m, h);
        typename W::Frag fq, fk, fv, fd, acc;
        typename W::Mat s, ds;
        p.load_keys(fk, k);
        p.load_rows(fq, q);
        p.load_keys(fv, v);
        p.load_rows(fd, dout);
        W::clear(s);
        W::clear(ds);
        w.scores(fk, fq, s);
        w.scores(fv, fd, ds);
        p.probabilities(s, stats);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            // delta = dout . out = sum of p dp
            float del = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) del = p.dead(t, j) ? del : __builtin_fmaf(s[t][n][j], ds[t][n][j], del);
            del = column_sum(del);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    ds[t][n][j] = p.dead(t, j) || !p.has_row(n) ? 0.0f : s[t][n][j] * (ds[t][n][j] - del);
        }
        if (dq != nullptr) {
            clear_own(acc);
            w.results(fk, ds, acc);
            p.store_rows(acc, a.scale, dq);
        }
        if (dv != nullptr) {
            w.exchange(s);
            clear_own(acc);
            w.results(fd, s, acc);
            p.store_keys(acc, 1.0f, dv);
        }
        if (dk == nullptr && db == nullptr) return;
        w.exchange(ds);
        if (db != nullptr) p.store_bias(ds, db);
        if (dk == nullptr) return;
        clear_own(acc);
        w.results(fq, ds, acc);
        p.store_keys(acc, a.scale, dk);
    });
}

template <int ND, int NT>
__global__ __launch_bounds__(256, NT < 3 && ND * NT <= 4 ? 2 : 1) void second_kernel(AttnArgs a, AttnSeconds x, float* go, float* gq, float* gk, float* gv,
                                                     float* gb)
{
    using W = Whole<ND, NT>;
    __shared__ __attribute__((aligned(16))) float lds[4][W::kFloats];
    const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
    const W w{m, h, lds[T::index()]};
    T::each_piece((int64_t)a.batch * a.kv_heads, whole_run(a), [&](int64_t piece) {
        const Problem<ND, NT> p(a, piece, m, h);
        typename W::Frag fq, fk, fv, fd, fvq, fvk, fvv, acc;
        typename W::Mat s, ds, gg, ee;
        p.load_keys(fk, x.k);
        p.load_rows(fq, x.q);
        p.load_rows(fvq, x.vq);
        p.load_keys(fvk, x.vk);
        p.load_rows(fd, x.dout);
        p.load_keys(fv, x.v);
        p.load_keys(fvv, x.vv);
        W::clear(s);
        W::clear(ds);
        W::clear(gg);
        W::clear(ee);
        w.scores(fk, fq, s);
        w.scores(fk, fvq, gg);
        w.scores(fvk, fq, gg);
        w.scores(fv, fd, ds);
        w.scores(fvv, fd, ee);
        p.probabilities(s, x.stats);
        float vterm[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float v = x.vbias != nullptr && p.term_m[t] != minus_inf()
                                ? x.vbias[p.b * x.vbias_b + (16 * t + m) * x.vbias_k]
                                : 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) vterm[t][j] = __shfl(v, 4 * h + j, 64);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float del = 0.0f, mean = 0.0f, sum = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    gg[t][n][j] = __builtin_fmaf(gg[t][n][j], a.scale, vterm[t][j]);
                    if (p.dead(t, j) || !p.has_row(n)) gg[t][n][j] = ds[t][n][j] = ee[t][n][j] = 0.0f;
                    del = __builtin_fmaf(s[t][n][j], ds[t][n][j], del);
                    mean = __builtin_fmaf(s[t][n][j], gg[t][n][j], mean);
                }
            del = column_sum(del);
            mean = column_sum(mean);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // T = G (dp - delta) - g dp + E
                    const float d = ds[t][n][j] - del;
                    const float v = __builtin_fmaf(-mean, ds[t][n][j], __builtin_fmaf(gg[t][n][j], d, ee[t][n][j]));
                    ee[t][n][j] = v;
                    sum = __builtin_fmaf(s[t][n][j], v, sum);
                    gg[t][n][j] = s[t][n][j] * (gg[t][n][j] - mean);   // H
                    ds[t][n][j] = s[t][n][j] * d;
                }
            sum = column_sum(sum);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) ee[t][n][j] = s[t][n][j] * (ee[t][n][j] - sum);   // U
        }
        if (go != nullptr) {
            clear_own(acc);
            w.results(fv, gg, acc);
            w.results(fvv, s, acc);
            p.store_rows(acc, 1.0f, go);
        }
        if (gq != nullptr) {
            clear_own(acc);
            w.results(fk, ee, acc);
            w.results(fvk, ds, acc);
            p.store_rows(acc, a.scale, gq);
        }
        if (gv != nullptr) {
            w.exchange(gg);
            clear_own(acc);
            w.results(fd, gg, acc);
            p.store_keys(acc, 1.0f, gv);
        }
        if (gk == nullptr && gb == nullptr) return;
        w.exchange(ee);
        if (gb != nullptr) p.store_bias(ee, gb);
        if (gk == nullptr) return;
        w.exchange(ds);
        clear_own(acc);
        w.results(fq, ee, acc);
        w.results(fvq, ds, acc);
        p.store_keys(acc, a.scale, gk);
    });
}

// f.template operator()<ND, NT>() for what attn_whole() takes.
template <class F>
void with_whole(const AttnArgs& a, F&& f)
{
    const int64_t n = a.rows > a.keys ? a.rows : a.keys;
    const auto tiles = [&]<int ND>() {
        if (n <= 16) return f.template operator()<ND, 1>();
        if (n <= 32) return f.template operator()<ND, 2>();
        return f.template operator()<ND, 3>();
    };
    if (a.dim <= 16)
        tiles.template operator()<1>();
    else if (a.dim <= 32)
        tiles.template operator()<2>();
    else if (a.dim <= 48)
        tiles.template operator()<3>();
    else
        tiles.template operator()<4>();
}

hipError_t join_bias(const AttnArgs& a, float* db, const float* partial, hipStream_t s)
{
    hipError_t e = hipGetLastError();
    AttnJoins joins{};
    if (a.kv_heads > 1) joins.add({a.batch, a.kv_heads, a.keys, partial, db});
    return e == hipSuccess ? launch_attn_joins(joins, s) : e;
}

unsigned whole_grid(const AttnArgs& a) { return T::grid((int64_t)a.batch * a.kv_heads, whole_run(a)); }

}  // namespace

// Both ways, us (forward; backward; second order), 2,000 x 8 heads: 32 x 32 x 32
// 66; 114; 234, by tiles 134; 407; 1,231. 46 x 46 x 64 262; 490; 1,306, by tiles
// 423; 1,060; 3,110. (The third tile of 16 does not fit the registers either in the
// second order of heads above 16 wide, and is the faster way all the same; a fourth
// was not tried.)
bool attn_whole(const AttnArgs& a) { return a.dim <= 64 && a.rows <= 48 && a.keys <= 48; }

hipError_t launch_whole_forward(const AttnArgs& a, emu_heads_t q, emu_heads_t k, emu_heads_t v, float* out, float* stats,
                                hipStream_t s)
{
    with_whole(a, [&]<int ND, int NT>() { forward_kernel<ND, NT><<<whole_grid(a), 256, 0, s>>>(a, q, k, v, out, stats); });
    return hipGetLastError();
}

hipError_t launch_whole_backward(const AttnArgs& a, emu_heads_t dout, emu_heads_t q, emu_heads_t k, emu_heads_t v,
                                 const float* stats, float* dq, float* dk, float* dv, float* dbias, float* partial,
                                 hipStream_t s)
{
    float* const to_b = dbias != nullptr && a.kv_heads > 1 ? partial : dbias;
    with_whole(a, [&]<int ND, int NT>() {
        backward_kernel<ND, NT><<<whole_grid(a), 256, 0, s>>>(a, dout, q, k, v, stats, dq, dk, dv, to_b);
    });
    return join_bias(a, dbias, partial, s);
}

hipError_t launch_whole_second(const AttnArgs& a, const AttnSeconds& x, float* gdout, float* gq, float* gk, float* gv,
                               float* gbias, float* partial, hipStream_t s)
{
    float* const to_b = gbias != nullptr && a.kv_heads > 1 ? partial : gbias;
    with_whole(a, [&]<int ND, int NT>() {
        second_kernel<ND, NT><<<whole_grid(a), 256, 0, s>>>(a, x, gdout, gq, gk, gv, to_b);
    });
    return join_bias(a, gbias, partial, s);
}

}  // namespace emu
