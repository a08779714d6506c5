// C ABI of the attention operators (declarations and full contract in
// include/emu_attention.h): argument checks, workspace layouts and the
// launches on the caller's stream.  Nothing is allocated here.
#include <hip/hip_runtime.h>

#include <cmath>

#include "emu_attn_launch.h"
#include "emu_block_launch.h"

namespace {

using emu::AttnArgs;
using emu::AttnPlan;

constexpr int64_t kMaxSize = (int64_t)1 << 30;

emu_status_t from_hip(hipError_t e)
{
    if (e == hipSuccess) return EMU_STATUS_SUCCESS;
    if (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation) return EMU_STATUS_ALLOC_FAILED;
    return EMU_STATUS_LAUNCH_FAILED;
}

hipStream_t stream_of(void* s) { return static_cast<hipStream_t>(s); }

bool bad_workspace(const void* ws, size_t have, size_t need)
{
    return need > 0 && (ws == nullptr || have < need || ((uintptr_t)ws & 255u) != 0);
}

bool on_gfx950()
{
    emu::DeviceInfo dev;
    return emu::api_current_device(dev);
}

// The call's sizes, checked.
emu_status_t args_of(const emu_attention_t* in, AttnArgs& a)
{
    if (in == nullptr || in->batch < 0 || in->queries < 0 || in->keys < 0 || in->heads < 0 || in->kv_heads < 0 ||
        in->dim < 1 || !std::isfinite(in->scale))
        return EMU_STATUS_INVALID_VALUE;
    if (in->heads > 0 && (in->kv_heads < 1 || in->heads % in->kv_heads != 0)) return EMU_STATUS_INVALID_VALUE;
    if (in->dim > EMU_ATTENTION_MAX_DIM || in->batch > kMaxSize || in->queries > kMaxSize || in->keys > kMaxSize ||
        in->queries * in->heads > kMaxSize)
        return EMU_STATUS_NOT_SUPPORTED;
    a = AttnArgs{};
    a.batch = (int)in->batch;
    a.queries = (int)in->queries;
    a.keys = (int)in->keys;
    a.heads = in->heads;
    a.kv_heads = in->heads > 0 ? in->kv_heads : 0;
    a.share = in->heads > 0 ? in->heads / in->kv_heads : 0;
    a.dim = in->dim;
    a.rows = in->queries * a.share;
    // (r times the inverse's excess, below share, has to stay below 2^32)
    if (a.share > 1 && a.rows <= ((int64_t)1 << 32) / a.share) a.share_inverse = (uint32_t)((((uint64_t)1 << 32) + a.share - 1) / a.share);
    a.scale = in->scale;
    a.bias = in->key_bias;
    a.bias_b = in->key_bias_batch;
    a.bias_k = in->key_bias_key;
    a.mask = in->key_mask;
    a.mask_b = in->key_mask_batch;
    a.mask_k = in->key_mask_key;
    a.lengths = in->lengths;
    a.lengths_64 = in->lengths_64;
    return EMU_STATUS_SUCCESS;
}

bool has_rows(const AttnArgs& a) { return a.batch > 0 && a.rows > 0; }
bool has_keys(const AttnArgs& a) { return a.batch > 0 && a.keys > 0 && a.kv_heads > 0; }

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Arrays one after the other in a workspace.
struct Layout {
    char* base;
    size_t bytes = 0;
    explicit Layout(void* p) : base(static_cast<char*>(p)) {}
    float* take(size_t floats)
    {
        if (floats == 0) return nullptr;
        float* at = base != nullptr ? reinterpret_cast<float*>(base + bytes) : nullptr;
        bytes += round256(floats * sizeof(float));
        return at;
    }
};

size_t rows_of(const AttnArgs& a) { return (size_t)a.batch * a.queries * a.heads; }

struct ForwardSpace {
    AttnPlan plan;
    float* partial;
    void* images;
    size_t bytes;
    ForwardSpace(const AttnArgs& a, void* ws) : plan(emu::attn_plan(a, emu::AttnPass::forward))
    {
        Layout l(ws);
        partial = l.take(emu::attn_forward_partial(a, plan));
        images = plan.images ? l.take(emu::attn_key_images(a, 2) / sizeof(float)) : nullptr;
        bytes = l.bytes;
    }
};
size_t forward_bytes(const AttnArgs& a)
{
    return !has_rows(a) || emu::attn_whole(a) ? 0 : ForwardSpace(a, nullptr).bytes;
}

struct BackwardSpace {
    AttnPlan rows, keys;
    float *delta, *dq, *dk, *dv, *db;
    void *key_images, *row_images;
    size_t bytes;
    BackwardSpace(const AttnArgs& a, void* ws) : rows(emu::attn_plan(a, emu::AttnPass::rows)), keys(emu::attn_plan(a, emu::AttnPass::keys))
    {
        Layout l(ws);
        delta = dq = dk = dv = db = nullptr;
        key_images = row_images = nullptr;
        if (emu::attn_whole(a)) {
            db = l.take(emu::attn_whole_partial(a));
            bytes = l.bytes;
            return;
        }
        delta = l.take(rows_of(a));
        dq = l.take(emu::attn_rows_partial(a, rows));
        dk = l.take(emu::attn_keys_partial(a, keys));
        dv = l.take(emu::attn_keys_partial(a, keys));
        db = l.take(emu::attn_bias_partial(a, keys));
        if (rows.images) key_images = l.take(emu::attn_key_images(a, 2) / sizeof(float));
        if (keys.images) row_images = l.take(emu::attn_row_images(a, 2) / sizeof(float));
        bytes = l.bytes;
    }
};

struct SecondSpace {
    AttnPlan rows, keys;
    float *delta, *sums, *go, *gq, *gk, *gv, *gb;
    void *key_images, *row_images;
    size_t bytes;
    SecondSpace(const AttnArgs& a, void* ws) : rows(emu::attn_plan(a, emu::AttnPass::second_rows)), keys(emu::attn_plan(a, emu::AttnPass::second_keys))
    {
        Layout l(ws);
        delta = sums = go = gq = gk = gv = gb = nullptr;
        key_images = row_images = nullptr;
        if (emu::attn_whole(a)) {
            gb = l.take(emu::attn_whole_partial(a));
            bytes = l.bytes;
            return;
        }
        delta = l.take(rows_of(a));
        sums = l.take(2 * rows.splits * rows_of(a));
        go = l.take(emu::attn_rows_partial(a, rows));
        gq = l.take(emu::attn_rows_partial(a, rows));
        gk = l.take(emu::attn_keys_partial(a, keys));
        gv = l.take(emu::attn_keys_partial(a, keys));
        gb = l.take(emu::attn_bias_partial(a, keys));
        if (rows.images) key_images = l.take(emu::attn_key_images(a, 4) / sizeof(float));
        if (keys.images) row_images = l.take(emu::attn_row_images(a, 3) / sizeof(float));
        bytes = l.bytes;
    }
};

// Zeros in the place of gradients that nothing reaches.
hipError_t zero(float* p, size_t floats, hipStream_t s)
{
    return p != nullptr && floats > 0 ? emu::launch_zero(p, (int64_t)floats, s) : hipSuccess;
}

emu_status_t zero_keys(const AttnArgs& a, float* dk, float* dv, float* dbias, hipStream_t s)
{
    const size_t n = (size_t)a.batch * a.keys * a.kv_heads * a.dim;
    hipError_t e = zero(dk, n, s);
    if (e == hipSuccess) e = zero(dv, n, s);
    if (e == hipSuccess) e = zero(dbias, (size_t)a.batch * a.keys, s);
    return from_hip(e);
}

}  // namespace

extern "C" {

int emu_attention_version(void) { return 100; }

// ---- attention -------------------------------------------------------------------

emu_status_t emu_cross_attention_workspace(const emu_attention_t* in, size_t* bytes)
{
    AttnArgs a;
    const emu_status_t st = args_of(in, a);
    if (st != EMU_STATUS_SUCCESS) return st;
    if (bytes == nullptr) return EMU_STATUS_INVALID_VALUE;
    *bytes = forward_bytes(a);
    return EMU_STATUS_SUCCESS;
}

emu_status_t emu_cross_attention(const emu_attention_t* in, emu_heads_t q, emu_heads_t k, emu_heads_t v, float* out,
                                 float* stats, void* workspace, size_t workspace_bytes, void* stream)
{
    AttnArgs a;
    const emu_status_t st = args_of(in, a);
    if (st != EMU_STATUS_SUCCESS) return st;
    if (has_rows(a) && (q.data == nullptr || out == nullptr)) return EMU_STATUS_INVALID_VALUE;
    if (has_keys(a) && (k.data == nullptr || v.data == nullptr)) return EMU_STATUS_INVALID_VALUE;
    if (!has_rows(a)) return EMU_STATUS_SUCCESS;
    if (bad_workspace(workspace, workspace_bytes, forward_bytes(a))) return EMU_STATUS_INVALID_VALUE;
    if (!on_gfx950()) return EMU_STATUS_NOT_SUPPORTED;
    if (emu::attn_whole(a)) return from_hip(emu::launch_whole_forward(a, q, k, v, out, stats, stream_of(stream)));
    const ForwardSpace w(a, workspace);
    const emu_heads_t keys[] = {k, v};
    hipError_t e = w.plan.images ? emu::launch_attn_images(a, 2, keys, w.images, 0, nullptr, nullptr, stream_of(stream)) : hipSuccess;
    if (e == hipSuccess) e = emu::launch_attn_forward(a, w.plan, q, k, v, w.images, out, stats, w.partial, stream_of(stream));
    return from_hip(e);
}

emu_status_t emu_cross_attention_backward_workspace(const emu_attention_t* in, size_t* bytes)
{
    AttnArgs a;
    const emu_status_t st = args_of(in, a);
    if (st != EMU_STATUS_SUCCESS) return st;
    if (bytes == nullptr) return EMU_STATUS_INVALID_VALUE;
    *bytes = has_rows(a) ? BackwardSpace(a, nullptr).bytes : 0;
    return EMU_STATUS_SUCCESS;
}

emu_status_t emu_cross_attention_backward(const emu_attention_t* in, emu_heads_t dout, emu_heads_t q, emu_heads_t k,
                                          emu_heads_t v, const float* out, const float* stats, float* dq, float* dk,
                                          float* dv, float* dbias, void* workspace, size_t workspace_bytes,
                                          void* stream)
{
    AttnArgs a;
    const emu_status_t st = args_of(in, a);
    if (st != EMU_STATUS_SUCCESS) return st;
    if (has_rows(a) && (dout.data == nullptr || q.data == nullptr || out == nullptr || stats == nullptr))
        return EMU_STATUS_INVALID_VALUE;
    if (has_keys(a) && (k.data == nullptr || v.data == nullptr)) return EMU_STATUS_INVALID_VALUE;
    const bool rows = has_rows(a), keys = a.batch > 0 && a.keys > 0;
    const bool keys_wanted = keys && (dk != nullptr || dv != nullptr || dbias != nullptr);
    if (!(rows && dq != nullptr) && !keys_wanted) return EMU_STATUS_SUCCESS;
    if (rows && bad_workspace(workspace, workspace_bytes, BackwardSpace(a, nullptr).bytes)) return EMU_STATUS_INVALID_VALUE;
    if (!on_gfx950()) return EMU_STATUS_NOT_SUPPORTED;
    const hipStream_t s = stream_of(stream);
    if (!rows) return zero_keys(a, dk, dv, dbias, s);
    const BackwardSpace w(a, workspace);
    if (emu::attn_whole(a))
        return from_hip(emu::launch_whole_backward(a, dout, q, k, v, stats, dq, dk, dv, dbias, w.db, s));
    const emu_heads_t key_side[] = {k, v}, row_side[] = {q, dout};
    emu::AttnJoins joins{};
    hipError_t e = emu::launch_attn_images(a, w.rows.images && dq != nullptr ? 2 : 0, key_side, w.key_images,
                                           w.keys.images && keys_wanted ? 2 : 0, row_side, w.row_images, s);
    if (e == hipSuccess)
        e = emu::launch_attn_backward_rows(a, w.rows, dout, q, k, v, out, stats, w.key_images, w.delta, dq, w.dq, joins, s);
    if (e == hipSuccess && keys_wanted)
        e = emu::launch_attn_backward_keys(a, w.keys, dout, q, k, v, w.row_images, stats, w.delta, dk, dv, dbias, w.dk, w.dv, w.db, joins, s);
    if (e == hipSuccess) e = emu::launch_attn_joins(joins, s);
    return from_hip(e);
}

emu_status_t emu_cross_attention_backward2_workspace(const emu_attention_t* in, size_t* bytes)
{
    AttnArgs a;
    const emu_status_t st = args_of(in, a);
    if (st != EMU_STATUS_SUCCESS) return st;
    if (bytes == nullptr) return EMU_STATUS_INVALID_VALUE;
    *bytes = has_rows(a) ? SecondSpace(a, nullptr).bytes : 0;
    return EMU_STATUS_SUCCESS;
}

emu_status_t emu_cross_attention_backward2(const emu_attention_t* in, emu_heads_t vq, emu_heads_t vk, emu_heads_t vv,
                                           const float* vbias, int64_t vbias_batch, int64_t vbias_key,
                                           emu_heads_t dout, emu_heads_t q, emu_heads_t k, emu_heads_t v,
                                           const float* out, const float* stats, float* gdout, float* gq, float* gk,
                                           float* gv, float* gbias, void* workspace, size_t workspace_bytes,
                                           void* stream)
{
    AttnArgs a;
    const emu_status_t st = args_of(in, a);
    if (st != EMU_STATUS_SUCCESS) return st;
    if (has_rows(a) && (dout.data == nullptr || q.data == nullptr || out == nullptr || stats == nullptr))
        return EMU_STATUS_INVALID_VALUE;
    if (has_keys(a) && (k.data == nullptr || v.data == nullptr)) return EMU_STATUS_INVALID_VALUE;
    const bool rows = has_rows(a), keys = a.batch > 0 && a.keys > 0;
    const bool rows_wanted = rows && (gdout != nullptr || gq != nullptr);
    const bool keys_wanted = keys && (gk != nullptr || gv != nullptr || gbias != nullptr);
    if (!rows_wanted && !keys_wanted) return EMU_STATUS_SUCCESS;
    if (rows && bad_workspace(workspace, workspace_bytes, SecondSpace(a, nullptr).bytes)) return EMU_STATUS_INVALID_VALUE;
    if (!on_gfx950()) return EMU_STATUS_NOT_SUPPORTED;
    const hipStream_t s = stream_of(stream);
    if (!rows) return zero_keys(a, gk, gv, gbias, s);
    const SecondSpace w(a, workspace);
    const emu::AttnSeconds x{vq, vk, vv, vbias, vbias_batch, vbias_key, dout, q, k, v, out, stats};
    if (emu::attn_whole(a)) return from_hip(emu::launch_whole_second(a, x, gdout, gq, gk, gv, gbias, w.gb, s));
    const emu_heads_t key_side[] = {k, v, vk, vv}, row_side[] = {q, dout, vq};
    emu::AttnJoins joins{};
    hipError_t e = emu::launch_attn_images(a, w.rows.images ? 4 : 0, key_side, w.key_images,
                                           w.keys.images && keys_wanted ? 3 : 0, row_side, w.row_images, s);
    if (e == hipSuccess) e = emu::launch_attn_second_sums(a, w.rows, x, w.key_images, w.delta, w.sums, s);
    if (e == hipSuccess && rows_wanted)
        e = emu::launch_attn_second_rows(a, w.rows, x, w.key_images, w.delta, w.sums, gdout, gq, w.go, w.gq, joins, s);
    if (e == hipSuccess && keys_wanted)
        e = emu::launch_attn_second_keys(a, w.keys, x, w.row_images, w.delta, w.sums, w.rows.splits, gk, gv, gbias, w.gk, w.gv, w.gb, joins, s);
    if (e == hipSuccess) e = emu::launch_attn_joins(joins, s);
    return from_hip(e);
}

// ---- rotary positions --------------------------------------------------------------

emu_status_t emu_rotary(int64_t batch, int64_t tokens, int64_t heads, int64_t dim, emu_heads_t x,
                        const int64_t* positions, int64_t positions_batch, int64_t positions_token,
                        const uint64_t* turns, int64_t pairs, emu_rotary_layout_t layout, float magnitude, int inverse,
                        float* y, void* stream)
{
    if (batch < 0 || tokens < 0 || heads < 0 || dim < 0 || pairs < 0 || pairs > dim / 2 ||
        ((int)layout != EMU_ROTARY_HALF && (int)layout != EMU_ROTARY_INTERLEAVED) || !std::isfinite(magnitude))
        return EMU_STATUS_INVALID_VALUE;
    if (batch > kMaxSize || tokens > kMaxSize || heads > kMaxSize || dim > EMU_ROTARY_MAX_DIM || heads * dim > kMaxSize)
        return EMU_STATUS_NOT_SUPPORTED;
    if (batch == 0 || tokens == 0 || heads == 0 || dim == 0) return EMU_STATUS_SUCCESS;
    if (x.data == nullptr || y == nullptr || (pairs > 0 && (positions == nullptr || turns == nullptr)))
        return EMU_STATUS_INVALID_VALUE;
    if (!on_gfx950()) return EMU_STATUS_NOT_SUPPORTED;
    const emu::RotaryArgs a{batch, tokens, (int)heads, (int)dim, (int)pairs, (int)layout, inverse != 0, x,
                            positions, positions_batch, positions_token, turns, magnitude, y};
    return from_hip(emu::launch_rotary(a, stream_of(stream)));
}

// ---- dropout -----------------------------------------------------------------------

emu_status_t emu_dropout(int64_t rows, int64_t cols, const float* x, int64_t ldx, double p, const int64_t* seed,
                         const float* residual, int64_t ldr, float* y, int64_t ldy, void* stream)
{
    const int64_t least = cols > 1 ? cols : 1;
    if (rows < 0 || cols < 0 || !(p >= 0.0 && p <= 1.0) || ldx < least || ldy < least ||
        (residual != nullptr && ldr < least))
        return EMU_STATUS_INVALID_VALUE;
    if (rows > 0 && cols > ((int64_t)1 << 60) / rows) return EMU_STATUS_NOT_SUPPORTED;
    if (rows == 0 || cols == 0) return EMU_STATUS_SUCCESS;
    if (x == nullptr || y == nullptr || seed == nullptr) return EMU_STATUS_INVALID_VALUE;
    if (!on_gfx950()) return EMU_STATUS_NOT_SUPPORTED;
    // p = 1 keeps nothing: its scale is of no element
    const emu::DropoutArgs a{rows, cols, x, ldx, (uint64_t)std::llrint(p * 4294967296.0),
                             p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f, seed, residual, ldr, y, ldy};
    return from_hip(emu::launch_dropout(a, stream_of(stream)));
}

}  // extern "C"
