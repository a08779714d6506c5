/*
 * emu_attention -- the operators of a transformer block's attention half, on
 * AMD MI355X (gfx950): attention of queries over keys of another length,
 * rotary positions, and dropout with the residual sum, beside the linears,
 * norms and feed-forward projections of emu_block.h.
 *
 * An interatomic potential lets the tokens of an atom's neighbours attend to
 * each other under a bias, the logarithm of the cutoff function; its forces
 * are the gradient of the energy, and training on forces differentiates that
 * gradient once more.  Attention therefore has a backward pass and that
 * pass's own backward pass; the other two operators are linear maps, whose
 * derivatives are the maps again (rotated back; the same mask).
 *
 * Conventions: those of emu_block.h (FP32 device arrays owned by the caller,
 * argument checks before any HIP call, nothing allocated, workspaces from the
 * caller, any pointer alignment of 4 bytes, asynchronous work on `stream`, no
 * atomics, sums in a fixed order, so the same call gives the same bits;
 * outputs may not overlap inputs unless said otherwise).  Inputs may overlap
 * each other.
 */
#ifndef EMU_ATTENTION_H
#define EMU_ATTENTION_H

#include "emu_sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of this header (major * 100 + minor). */
int emu_attention_version(void);

/* ---- attention ---------------------------------------------------------------
 *
 * For sequence b, query i and head h (key and value head h / (heads /
 * kv_heads), written k_j, v_j):
 *   t_j = scale * (q_i . k_j) + key_bias_j,   p = softmax over j of t,
 *   out_i = sum over j of p_j v_j.
 * Key j takes part if j < lengths[b] (all do without lengths; what is below 0
 * or above `keys` counts as these), key_mask is not 0 there (all do without),
 * and key_bias is not -infinity there.  What the others' keys and values hold
 * is not used (they may be infinite or NaN).  A row without keys gives zeros,
 * and has no gradients.
 *
 * An array of [batch][token][head][dim] floats, read in place: element (b, t,
 * h, d) is data[b * batch + t * token + h * head + d].  Strides may be 0 (and
 * negative).
 */
typedef struct {
    const float* data;
    int64_t batch, token, head;
} emu_heads_t;

typedef struct {
    int64_t batch, queries, keys;
    int32_t heads, kv_heads, dim;          /* heads a multiple of kv_heads */
    float scale;
    const float* key_bias;                 /* element (b, j) at b * key_bias_batch + j * key_bias_key; or NULL */
    int64_t key_bias_batch, key_bias_key;
    const uint8_t* key_mask;               /* likewise; or NULL */
    int64_t key_mask_batch, key_mask_key;
    const void* lengths;                   /* `batch` int32_t, or int64_t where lengths_64; or NULL */
    int32_t lengths_64;
} emu_attention_t;

#define EMU_ATTENTION_MAX_DIM 128

/*
 * out: [batch][queries][heads][dim], dense.  stats: [batch][queries][heads][2]
 * receives what the backward passes need of each row's softmax, or NULL.
 *
 * Products run on the FP32 matrix instruction where sequences are short (up to
 * 48 keys and 48 rows of a key head, queries times the heads that share it;
 * heads up to 64 wide) and in the forward pass of up to 16 rows; elsewhere on
 * BF16 pieces of the operands, six products down to 2^-16 each, which leave out
 * less than 2^-24 of a product, FP32's own rounding (more of a factor below
 * 2^-110, whose lowest pieces BF16 does not hold).  There an infinite element
 * of a query or of a key or value that takes part gives NaN.  Running maxima,
 * sums and outputs are held in FP32, the outputs before they are divided by the
 * weights' sum: values above 2^126 / keys in size may pass FP32's range there.
 *
 * batch, queries or heads 0: nothing is done; keys == 0: zeros.
 * Errors: EMU_STATUS_INVALID_VALUE for a negative size, dim < 1, kv_heads < 1
 * while heads > 0, heads not a multiple of kv_heads, a scale that is not
 * finite, NULL arrays that have elements, a short or misaligned (256 bytes)
 * workspace; EMU_STATUS_NOT_SUPPORTED for dim > EMU_ATTENTION_MAX_DIM, batch,
 * queries * heads or keys above 2^30, or a device that is not gfx950.
 *
 * Workspaces (of all three calls): ask for each call's own struct.  The bytes
 * go by its sizes and by whether lengths is NULL (by nothing else that it
 * points to), since both decide into how many ranges the work is cut, and they
 * do not grow evenly with any size: a smaller batch, shorter sequences or the
 * same sizes with lengths may need more.  A workspace that serves several
 * calls has to hold the most that any of their structs asks for.
 */
emu_status_t emu_cross_attention_workspace(const emu_attention_t* a, size_t* bytes);
emu_status_t emu_cross_attention(const emu_attention_t* a, emu_heads_t q, emu_heads_t k, emu_heads_t v,
                                 float* out, float* stats, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * Gradients from dout, with out and stats as the forward call wrote them
 * (dense), dp_j = dout . v_j, delta = dout . out, ds = p (dp - delta):
 *   dq = scale sum over j of ds k_j    ([batch][queries][heads][dim], dense)
 *   dk = scale sum over rows of ds q,  dv = sum over rows of p dout
 *                                      ([batch][keys][kv_heads][dim], dense)
 *   dbias = sum over rows and heads of ds   ([batch][keys], dense)
 * Each of the four may be NULL.  Keys that do not take part get zeros.
 */
emu_status_t emu_cross_attention_backward_workspace(const emu_attention_t* a, size_t* bytes);
emu_status_t emu_cross_attention_backward(const emu_attention_t* a, emu_heads_t dout, emu_heads_t q,
                                          emu_heads_t k, emu_heads_t v, const float* out,
                                          const float* stats, float* dq, float* dk, float* dv,
                                          float* dbias, void* workspace, size_t workspace_bytes,
                                          void* stream);

/*
 * Gradients of the backward pass: for a scalar L with vq = dL/d(dq), vk =
 * dL/d(dk), vv = dL/d(dv) and vbias = dL/d(dbias) (element (b, j) at b *
 * vbias_batch + j * vbias_key); data NULL, or vbias NULL, stands for zeros:
 *   G = scale (vq . k_j + q . vk_j) + vbias_j,  g = sum of p G,  H = p (G - g),
 *   T = G (dp - delta) - g dp + dout . vv_j,     U = p (T - sum of p T),
 *   gdout = sum over j of H v_j + p vv_j,   gq = scale sum over j of U k_j + ds vk_j,
 *   gk = scale sum over rows of U q + ds vq,  gv = sum over rows of H dout,
 *   gbias = sum over rows and heads of U;
 * shapes as the forward and backward calls', each may be NULL.
 */
emu_status_t emu_cross_attention_backward2_workspace(const emu_attention_t* a, size_t* bytes);
emu_status_t emu_cross_attention_backward2(const emu_attention_t* a, emu_heads_t vq, emu_heads_t vk,
                                           emu_heads_t vv, const float* vbias, int64_t vbias_batch,
                                           int64_t vbias_key, emu_heads_t dout, emu_heads_t q,
                                           emu_heads_t k, emu_heads_t v, const float* out,
                                           const float* stats, float* gdout, float* gq, float* gk,
                                           float* gv, float* gbias, void* workspace,
                                           size_t workspace_bytes, void* stream);

/* ---- rotary positions -----------------------------------------------------------
 *
 * Rotates pairs of each head's first 2 * pairs elements by angles that grow
 * with the token's position; the rest of the head is copied.  Pair i is
 * (2 i, 2 i + 1) (EMU_ROTARY_INTERLEAVED) or (i, i + pairs) (EMU_ROTARY_HALF):
 *   a' = magnitude (a cos - b sin),  b' = magnitude (a sin + b cos),
 * angle = position * turns[i] * 2^-64 turns.  turns holds the frequencies as
 * 64-bit fractions of a turn, so that the product, taken modulo 2^64, is the
 * angle without whole turns, exactly, at any position (negative ones too).
 * inverse: by the opposite angle, which is also the gradient.
 * Cosines and sines are good to 2^-23.
 *
 * x: [batch][tokens][heads][dim] as above; positions: int64, element (b, t)
 * at b * positions_batch + t * positions_token; y: dense.  y may be x where x
 * is dense.
 * Errors: EMU_STATUS_INVALID_VALUE for a negative size, 2 * pairs > dim, a
 * bad layout, NULL arrays that have elements, a magnitude that is not finite;
 * EMU_STATUS_NOT_SUPPORTED for batch, tokens or heads * dim above 2^30, dim
 * above EMU_ROTARY_MAX_DIM, or a device that is not gfx950.
 */
#define EMU_ROTARY_MAX_DIM 65536

typedef enum {
    EMU_ROTARY_HALF = 0,
    EMU_ROTARY_INTERLEAVED = 1
} emu_rotary_layout_t;

emu_status_t emu_rotary(int64_t batch, int64_t tokens, int64_t heads, int64_t dim, emu_heads_t x,
                        const int64_t* positions, int64_t positions_batch, int64_t positions_token,
                        const uint64_t* turns, int64_t pairs, emu_rotary_layout_t layout,
                        float magnitude, int inverse, float* y, void* stream);

/* ---- dropout ----------------------------------------------------------------------
 *
 *   y = (kept ? x * scale : 0) + residual,  scale = FP32(1 / (1 - p)).
 * Element e (row * cols + col) is kept if word e % 4 of Philox4x32-10 (J. K.
 * Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", SC 2011) with
 * key seed[0] and the 128-bit counter e / 4 + 2^64 seed[1] is not below p
 * 2^32, rounded to the nearest whole number.  The mask is never stored: the
 * backward pass is the same call on the gradient, without the residual.
 *
 * seed: two int64 in device memory, read when the kernel runs (so a captured
 * call takes what is there when it is replayed).  residual: rows x cols or
 * NULL.  y may be x or residual where their leading dimensions are equal.
 * Errors: EMU_STATUS_INVALID_VALUE for a negative size, a leading dimension <
 * cols, p outside 0..1 or NaN, NULL arrays that have elements (seed too);
 * EMU_STATUS_NOT_SUPPORTED for more than 2^60 elements, or a device that is
 * not gfx950.
 */
emu_status_t emu_dropout(int64_t rows, int64_t cols, const float* x, int64_t ldx, double p,
                         const int64_t* seed, const float* residual, int64_t ldr, float* y,
                         int64_t ldy, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EMU_ATTENTION_H */
