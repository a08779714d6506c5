// Keys' and rows' arrays split beforehand for the attention of longer sequences
// (emu_attn_split.h): images of their tiles of 32 rows in LDS. Where several
// teams stream the same side this takes the splitting, the strides, odd widths
// and ends, and the keys that take no part out of their loops, which copy the
// images as they are.
//
// Bound by memory: 4 bytes read and 6 written per element; 2 x 16 heads of
// 4,096 keys and values of 64 (168 MB) in 32 us, 5.2 TB/s.
#include "emu_attn_split.h"

namespace emu {
namespace {

// The arrays of both sides, the keys' first.
struct ImageArrays {
    emu_heads_t of[7];
    int keys, all;
    int64_t key_tiles, row_tiles;   // per sequence and key head
    char *to_keys, *to_rows;
};

// A workgroup makes one array's part of an image, eight elements a thread.
template <int KS>
__global__ __launch_bounds__(kAttnTile * 4 * KS) void images_kernel(AttnArgs a, ImageArrays x)
{
    constexpr int RS = 32 * KS;
    const int n = blockIdx.y;
    const bool is_key = n < x.keys;
    emu_heads_t from = x.of[0];   // (chosen, not indexed: arguments stay in scalar registers)
#pragma unroll
    for (int i = 1; i < 7; ++i)
        if (n == i) from = x.of[i];
    const int64_t tiles = is_key ? x.key_tiles : x.row_tiles, all = (int64_t)a.batch * a.kv_heads * tiles;
    const int row = threadIdx.x / (RS / 8), col = threadIdx.x % (RS / 8) * 8;
    for (int64_t tile = blockIdx.x; tile < all; tile += gridDim.x) {
        const int64_t head = tile / tiles, r = (tile - head * tiles) * kAttnTile + row;
        const int b = (int)(head / a.kv_heads), g = (int)(head - (int64_t)b * a.kv_heads);
        const int limit = is_key ? keys_of(a, b) : 0;
        if (is_key && r - row >= limit) continue;   // (not read)
        f32x4_t u = {}, v = {};
        if (col < a.dim && from.data != nullptr) {
            if (is_key ? r < a.keys && key_term(a, b, (int)r, limit) != minus_inf() : r < a.rows) {
                const float* const p = is_key ? key_ptr(from, b, g, r) : row_ptr(from, b, row_at(a, g, r));
                u = load4(p, col, a.dim);
                v = load4(p, col + 4, a.dim);
            }
        }
        const Split8 s = split8<true>(u, v);
        char* const image = is_key ? x.to_keys + tile * attn_image_bytes(32 * KS, x.keys)
                                   : x.to_rows + tile * attn_image_bytes(32 * KS, x.all - x.keys);
        uint16_t* const to = reinterpret_cast<uint16_t*>(image) + ((is_key ? n : n - x.keys) * 3 * kAttnTile + row) * RS +
                             8 * (col / 8 ^ attn_image_place(KS, row));
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8_t*>(to + p * kAttnTile * RS) = s.p[p];
    }
}

template <int KS>
void launch_images(const AttnArgs& a, const ImageArrays& x, hipStream_t s)
{
    const int64_t tiles = x.key_tiles > x.row_tiles ? x.key_tiles : x.row_tiles, all = (int64_t)a.batch * a.kv_heads * tiles;
    images_kernel<KS><<<dim3((unsigned)(all < 65536 ? all : 65536), x.all), kAttnTile * 4 * KS, 0, s>>>(a, x);
}

int64_t tiles_of(int64_t n) { return (n + kAttnTile - 1) / kAttnTile; }

}  // namespace

size_t attn_key_images(const AttnArgs& a, int n)
{
    return (size_t)a.batch * a.kv_heads * tiles_of(a.keys) * attn_image_bytes(a.dim, n);
}
size_t attn_row_images(const AttnArgs& a, int m)
{
    return (size_t)a.batch * a.kv_heads * tiles_of(a.rows) * attn_image_bytes(a.dim, m);
}

hipError_t launch_attn_images(const AttnArgs& a, int n, const emu_heads_t* keys, void* key_images, int m,
                              const emu_heads_t* rows, void* row_images, hipStream_t s)
{
    ImageArrays x{};
    for (int i = 0; i < n; ++i) x.of[i] = keys[i];
    for (int i = 0; i < m; ++i) x.of[n + i] = rows[i];
    x.keys = n;
    x.all = n + m;
    x.key_tiles = n > 0 ? tiles_of(a.keys) : 0;
    x.row_tiles = m > 0 ? tiles_of(a.rows) : 0;
    x.to_keys = static_cast<char*>(key_images);
    x.to_rows = static_cast<char*>(row_images);
    if (x.all == 0 || x.key_tiles + x.row_tiles == 0) return hipSuccess;
    if (a.dim <= 32)
        launch_images<1>(a, x, s);
    else if (a.dim <= 64)
        launch_images<2>(a, x, s);
    else if (a.dim <= 96)
        launch_images<3>(a, x, s);
    else
        launch_images<4>(a, x, s);
    return hipGetLastError();
}

}  // namespace emu
