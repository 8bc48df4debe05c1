// xp_kv_dev.h — the 4-bit key/value cache: geometry, layout and codec shared by
// the cache operators (xp_kv.hip) and decode attention (xp_attn.hip).
//
// A cache is n_pages pages of `page` positions; a page holds, for every kv head
// in turn, page / 64 tiles of 64 positions. With NG = head_dim / 32 groups of 32
// values a tile is NG * 2176 bytes (4.25 bits a value):
//   K codes   16-byte chunk (pos, g) at g*1024 + pos*16, byte b = values 2b (low
//             nibble) and 2b + 1 of group g: the packed weights' chunk. A lane of
//             the score product takes one chunk, so its values share one scale.
//   K scales  byte (pos, g) at NG*1024 + g*64 + (pos%16)*4 + pos/16: the four
//             16-position blocks a lane works on are one dword.
//   V codes   8-byte chunk (pos, h) at NG*1088 + h*512 + pos*8, h = 16 values:
//             the row of a 4-bit transposing LDS read; consecutive positions are
//             consecutive 8-byte words, so those reads meet no bank twice.
//   V scales  byte (pos, g) at NG*2112 + g*64 + (pos/4%4)*16 + (pos/16)*4 + pos%4:
//             the 16 positions a lane holds probabilities of are 16 bytes in order.
#pragma once

#include "xp_common.h"

namespace xp {
namespace kv {

constexpr int kTilePos = 64;

struct Geo {
    int kv_heads;
    int groups;      // head_dim / 32
    int page;        // positions per page
    int n_pages;
    int max_pages;   // columns of the page table
};

__host__ __device__ __forceinline__ int tile_bytes(int groups) { return groups * 2176; }

// Where position pos (0 <= pos < max_pages * page) of a sequence lies: the byte
// offset of its tile, or -1 when its page is not one of the cache's.
__device__ __forceinline__ long long tile_at(const Geo& g, const int32_t* table_row, int head, int pos) {
    const int col = pos / g.page;
    const int id = table_row[col];
    if ((unsigned)id >= (unsigned)g.n_pages) return -1;
    const int tiles = g.page / kTilePos;
    return (((long long)id * g.kv_heads + head) * tiles + (pos - col * g.page) / kTilePos) * tile_bytes(g.groups);
}

__device__ __forceinline__ int k_code(int groups, int pos, int g) { return g * 1024 + pos * 16; }
__device__ __forceinline__ int k_scale(int groups, int pos, int g) {
    return groups * 1024 + g * 64 + (pos & 15) * 4 + (pos >> 4);
}
__device__ __forceinline__ int v_code(int groups, int pos, int h) { return groups * 1088 + h * 512 + pos * 8; }
__device__ __forceinline__ int v_scale(int groups, int pos, int g) {
    return groups * 2112 + g * 64 + ((pos >> 2) & 3) * 16 + (pos >> 4) * 4 + (pos & 3);
}

// The first position that a row at position `at` sees: any window up to 2^31 - 1, any at.
__device__ __forceinline__ int first_seen(int at, int window) {
    return window > 0 && at >= window ? at - window + 1 : 0;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0); }

// The smallest E4M3FN scale s with 6 s >= amax (amax >= 0), 448 when there is
// none, the NaN byte when amax is not finite. amax / 6 in fp32 places s within a
// step; six times an E4M3 value is exact, so the comparisons decide it exactly.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const float r = amax * (1.0f / 6.0f);
    int code = r >= 0x1p-6f ? (int)(__float_as_uint(r) >> 20) - ((127 - 7) << 3) : (int)(r * 512.0f);
    code = code > 0x7e ? 0x7e : code;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (code < 0x7e && 6.0f * e4m3_value((uint32_t)code) < amax) ++code;
    return (__float_as_uint(amax) & 0x7f800000u) == 0x7f800000u ? 0x7fu : (uint32_t)code;
}

// Eight e2m1 codes nearest to x / s, ties to the even code, beyond 6 s to 6 s; inv is
// 1 / s. The quotient is corrected once by its exact remainder and so rounded to the
// nearest fp32 number, which never crosses a midpoint of e2m1: a midpoint M times s is
// an fp32 number, and x next to it lies 2^-23 / p away relative to it (p < 2 its
// significand), more than half a step of M's, 2^-24 / m with M's significand m >= 1. A
// quotient that is M itself comes out as M. The conversion rounds to nearest even.
__device__ __forceinline__ uint32_t e2m1_codes(const float x[8], float s, float inv) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = x[i] * inv;
        const float c = __builtin_fmaf(__builtin_fmaf(-q, s, x[i]), inv, q);
        r[i] = __uint_as_float(__float_as_uint(c) | (__float_as_uint(x[i]) & 0x80000000u));   // -0 keeps its sign
    }
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[0], r[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[2], r[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[4], r[5], 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[6], r[7], 1.0f, 3);
}

inline bool geo_ok(const xp_kv_dims* d) {
    return d->kv_heads >= 1 && d->kv_heads <= 1024 && (d->head_dim == 64 || d->head_dim == 128 || d->head_dim == 256) &&
           d->page >= kTilePos && d->page % kTilePos == 0 && d->page <= (1 << 20) && d->n_pages >= 1;
}

// Shared checks of the calls that take a page table.
inline int check_geo(const xp_kv_dims* d, int32_t batch, int32_t max_pages) {
    if (!d) return XP_ERR_NULL;
    if (!geo_ok(d) || batch < 0 || batch > 65535 || max_pages < 1) return XP_ERR_SHAPE;
    if ((long long)max_pages * d->page > 0x7fffffffLL - 1024) return XP_ERR_SHAPE;
    return XP_OK;
}

inline Geo geo_of(const xp_kv_dims* d, int32_t max_pages) {
    return Geo{d->kv_heads, d->head_dim / 32, d->page, d->n_pages, max_pages};
}

// scale * log2(e), kept a normal number: neither 0 nor infinity may meet a masked -inf or a score of 0.
inline float log2_scale(float scale) {
    const double x = (double)scale * 1.4426950408889634;
    return (float)(x < 0x1p-126 ? 0x1p-126 : (x > 0x1p127 ? 0x1p127 : x));
}

// n rows of a buffer, `width` bytes each and `step` bytes apart (host).
struct Rows {
    const void* p;
    int64_t n, step, width;
    bool same(const Rows& o) const { return p == o.p && (step == o.step || n <= 1); }
};
// Whether two buffers' rows share a byte. Views into one wider buffer interleave without
// sharing any; with one step the shift between rows decides it, otherwise a walk over both.
inline bool rows_meet(const Rows& a, const Rows& b) {
    typedef __int128 wide;
    if (a.n < 1 || b.n < 1) return false;
    const wide a0 = (wide)(uintptr_t)a.p, b0 = (wide)(uintptr_t)b.p, d = b0 - a0;
    if (d >= (wide)(a.n - 1) * a.step + a.width || -d >= (wide)(b.n - 1) * b.step + b.width) return false;
    if (a.step == b.step) {
        // rows i of a and j of b meet where -b.width < d + (j - i) step < a.width
        const auto floor_div = [](wide x, wide y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };
        const wide lo = floor_div(-b.width - d, a.step) + 1, hi = -floor_div(d - a.width, a.step) - 1;
        return (lo > 1 - a.n ? lo : 1 - a.n) <= (hi < b.n - 1 ? hi : b.n - 1);
    }
    int64_t i = 0, j = 0;
    while (i < a.n && j < b.n) {
        const wide x = a0 + (wide)i * a.step, y = b0 + (wide)j * b.step;
        if (x + a.width <= y)
            i += (int64_t)((y - x - a.width) / a.step) + 1;
        else if (y + b.width <= x)
            j += (int64_t)((x - y - b.width) / b.step) + 1;
        else
            return true;
    }
    return false;
}

inline bool aligned_to(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace kv
}  // namespace xp
