// xp_attn_dev.h — what decode attention (xp_attn.hip) and attention over selected blocks
// (xp_attn_sparse.hip) share: a wave's view of one tile of the 4-bit cache for 16 query rows.
// Lane (c, q) = (lane % 16, lane / 16); see xp_attn.hip for the order of positions.
#pragma once

#include "xp_kv_dev.h"

namespace xp {
namespace attn {

typedef __attribute__((ext_vector_type(2))) _Float16 h16x2;
typedef __attribute__((ext_vector_type(8))) _Float16 h16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;

constexpr float kLift = 15.0f;   // exponentials are held as 2^kLift p: 2^15 is fp16's largest power of two

__device__ __forceinline__ float max_over_q(float x) {
    uint32_t u = __float_as_uint(x);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    u = __float_as_uint(x);
    auto b = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_q(float x) {
    uint32_t u = __float_as_uint(x);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    u = __float_as_uint(x);
    auto b = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ h16x8 frag(h16x2 a, h16x2 b, h16x2 c, h16x2 d) {
    return h16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Eight e2m1 codes times their scale (two values a pair, or one for all), exact.
__device__ __forceinline__ h16x8 decode8(uint32_t w, h16x2 s0, h16x2 s1, h16x2 s2, h16x2 s3) {
    return frag(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s0, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s1,
                __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s3);
}

template <int D>
struct Dim {
    static constexpr int NG = D / 32;          // groups
    static constexpr int NW = D / 32;          // dwords of K codes a lane holds of each position: D/8 dwords over 4 lanes
    static constexpr int NH = D / 16;          // 16-value columns of V
    static constexpr int VD = D / 8;           // dwords of V codes a lane copies
    static constexpr int kVBytes = 64 * D / 2; // V codes of a tile
};

// The 8 dims that dword w of lane quarter q covers.
template <int D>
__device__ __forceinline__ int dims_of(int q, int w) {
    if constexpr (D == 64) return 16 * q + 8 * w;
    return 128 * (w >> 2) + 32 * q + 8 * (w & 3);
}

// K codes and scales of a tile as a lane of the score product holds them.
template <int D>
struct KTile {
    uint32_t w[4][Dim<D>::NW];
    uint32_t s[D == 256 ? 2 : 1];
};
template <int D>
__device__ __forceinline__ void load_k(KTile<D>& k, const uint8_t* t, int c, int q) {
    constexpr int NG = Dim<D>::NG;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int pos = 16 * b + c;
        if constexpr (D == 64) {
            const uint2 v = *(const uint2*)(t + (q >> 1) * 1024 + pos * 16 + (q & 1) * 8);
            k.w[b][0] = v.x;
            k.w[b][1] = v.y;
        } else {
#pragma unroll
            for (int j = 0; j < NG / 4; ++j) {
                const uint4 v = *(const uint4*)(t + (4 * j + q) * 1024 + pos * 16);
                k.w[b][4 * j] = v.x;
                k.w[b][4 * j + 1] = v.y;
                k.w[b][4 * j + 2] = v.z;
                k.w[b][4 * j + 3] = v.w;
            }
        }
    }
    if constexpr (D == 64) {
        k.s[0] = *(const uint32_t*)(t + NG * 1024 + (q >> 1) * 64 + c * 4);
    } else {
#pragma unroll
        for (int j = 0; j < NG / 4; ++j) k.s[j] = *(const uint32_t*)(t + NG * 1024 + (4 * j + q) * 64 + c * 4);
    }
}
// Fragment w of block b: its eight codes times the scale of position 16 b + c.
template <int D>
__device__ __forceinline__ h16x8 k_frag(const KTile<D>& k, int b, int w) {
    const uint32_t sd = k.s[D == 256 ? w >> 2 : 0];
    const h16x2 p = b < 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sd, 1.0f, false)
                          : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sd, 1.0f, true);
    const _Float16 s = b & 1 ? p.y : p.x;
    const h16x2 ss = h16x2{s, s};
    return decode8(k.w[b][w], ss, ss, ss, ss);
}

// Four outputs to 16 bits, nearest even.
template <bool BF16>
__device__ __forceinline__ uint2 to16(f32x4 v) {
    if constexpr (BF16) {
        typedef __attribute__((ext_vector_type(4))) __bf16 b16x4;
        return __builtin_bit_cast(uint2, __builtin_convertvector(v, b16x4));
    } else {
        typedef __attribute__((ext_vector_type(4))) _Float16 h16x4;
        return __builtin_bit_cast(uint2, __builtin_convertvector(v, h16x4));
    }
}

}  // namespace attn
}  // namespace xp
