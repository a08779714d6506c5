// Keys' and rows' arrays split beforehand for the attention of longer sequences
// (emu_attn_split.h): images of their tiles of 32 rows in LDS. Where several
// teams stream the same side this takes the splitting, the strides, odd widths
// and ends, and the keys that take no part out of their loops, which copy the
// images as they are.
//
// Bound by memory: 4 bytes read and 6 to 7.5 written per element.
#include "emu_attn_split.h"

namespace emu {
namespace {

struct ImageArrays {
    emu_heads_t of[4];
    int n;
    int64_t tiles;       // per sequence and key head
    char* to;
};

// One workgroup per tile: the keys' tiles, then the rows'.
template <int KS>
__global__ __launch_bounds__(256) void images_kernel(AttnArgs a, ImageArrays keys, ImageArrays rows)
{
    constexpr int RS = 32 * KS + 8, GROUPS = kAttnTile * 4 * KS;   // of eight elements
    const int64_t heads = (int64_t)a.batch * a.kv_heads, key_tiles = keys.n > 0 ? heads * keys.tiles : 0;
    const int64_t all = key_tiles + (rows.n > 0 ? heads * rows.tiles : 0);
    for (int64_t tile = blockIdx.x; tile < all; tile += gridDim.x) {
        const bool is_key = tile < key_tiles;
        const ImageArrays& x = is_key ? keys : rows;
        const int64_t mine = is_key ? tile : tile - key_tiles, head = mine / x.tiles, first = (mine - head * x.tiles) * kAttnTile;
        const int b = (int)(head / a.kv_heads), g = (int)(head - (int64_t)b * a.kv_heads);
        const int limit = keys_of(a, b);
        uint16_t* const image = reinterpret_cast<uint16_t*>(x.to + mine * attn_image_bytes(32 * KS, x.n));
        for (int i = threadIdx.x; i < GROUPS; i += 256) {
            const int row = i / (4 * KS), col = i % (4 * KS) * 8;
            const int64_t r = first + row;
            const bool there = col < a.dim && (is_key ? r < a.keys && key_term(a, b, (int)r, limit) != minus_inf() : r < a.rows);
            const RowAt at = is_key ? RowAt{0, 0} : row_at(a, g, there ? r : 0);
            for (int n = 0; n < x.n; ++n) {
                f32x4_t u = {}, v = {};
                if (there && x.of[n].data != nullptr) {
                    const float* const p = is_key ? key_ptr(x.of[n], b, g, r) : row_ptr(x.of[n], b, at);
                    u = load4(p, col, a.dim);
                    v = load4(p, col + 4, a.dim);
                }
                const Split8 s = split8<true>(u, v);
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<bf16x8_t*>(image + ((n * 3 + p) * kAttnTile + row) * RS + col) = s.p[p];
            }
        }
    }
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
    ImageArrays k{}, r{};
    for (int i = 0; i < n; ++i) k.of[i] = keys[i];
    for (int i = 0; i < m; ++i) r.of[i] = rows[i];
    k.n = n;
    r.n = m;
    k.tiles = tiles_of(a.keys);
    r.tiles = tiles_of(a.rows);
    k.to = static_cast<char*>(key_images);
    r.to = static_cast<char*>(row_images);
    const int64_t all = (int64_t)a.batch * a.kv_heads * ((n > 0 ? k.tiles : 0) + (m > 0 ? r.tiles : 0));
    if (all == 0) return hipSuccess;
    const unsigned grid = (unsigned)(all < 65536 ? all : 65536);
    if (a.dim <= 32)
        images_kernel<1><<<grid, 256, 0, s>>>(a, k, r);
    else if (a.dim <= 64)
        images_kernel<2><<<grid, 256, 0, s>>>(a, k, r);
    else if (a.dim <= 96)
        images_kernel<3><<<grid, 256, 0, s>>>(a, k, r);
    else
        images_kernel<4><<<grid, 256, 0, s>>>(a, k, r);
    return hipGetLastError();
}

}  // namespace emu
