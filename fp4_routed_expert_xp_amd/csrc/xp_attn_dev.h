// xp_attn_dev.h — a wave's view of one tile of the 4-bit cache for 16 query rows. Decode attention
// (xp_attn.hip) takes the keys, their decoding and the rounding of outputs from here, and has steps
// for values, softmax and joins of its own, for one or two sixteens of rows; attention over chosen
// blocks (xp_attn_sparse.hip) and the few rows of a sequence in a mixed step (xp_attn_chunk.hip)
// share all of it. Lane (c, q) = (lane % 16, lane / 16); order of positions and precision are
// decode's: see xp_attn.hip.
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

// ---- a tile by steps, for 16 rows; row c of the lane's column

// The row at p (if it is there) as fp16 fragments; returns its score factor, scale_m * 2^scale_e
// being the scale in log2 units.
template <int D, bool BF16>
__device__ __forceinline__ float row_frags(const uint16_t* p, bool there, int q, float scale_m, int scale_e, h16x8 (&qf)[Dim<D>::NW]) {
    uint4 v[Dim<D>::NW];
#pragma unroll
    for (int w = 0; w < Dim<D>::NW; ++w) v[w] = there ? *(const uint4*)(p + dims_of<D>(q, w)) : uint4{0, 0, 0, 0};
    int k = 0;
    if constexpr (BF16) {
        uint32_t top = 0;                      // exponent field of the row's largest magnitude
#pragma unroll
        for (int w = 0; w < Dim<D>::NW; ++w) {
            const uint32_t u[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = (u[i] >> 7) & 255u, hi = (u[i] >> 23) & 255u;
                top = lo > top ? lo : top;
                top = hi > top ? hi : top;
            }
        }
        const int e = (int)max_over_q((float)top);
        // largest magnitude to [2^14, 2^15); rows with an infinity or NaN are left as they are
        k = e == 255 ? 0 : 141 - e;
        k = k > 100 ? 100 : k;
        const float up = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
        for (int w = 0; w < Dim<D>::NW; ++w) {
            const uint32_t u[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                qf[w][2 * i] = (_Float16)(__uint_as_float(u[i] << 16) * up);
                qf[w][2 * i + 1] = (_Float16)(__uint_as_float(u[i] & 0xffff0000u) * up);
            }
        }
    } else {
#pragma unroll
        for (int w = 0; w < Dim<D>::NW; ++w) qf[w] = __builtin_bit_cast(h16x8, v[w]);
    }
    // kept a normal number: a masked -inf times 0, or a score of 0 times infinity, would be NaN
    return fminf(fmaxf(__builtin_amdgcn_ldexpf(scale_m, scale_e - k), 0x1p-126f), 0x1p127f);
}

// V codes and scales of a tile as a lane copies them.
template <int D>
struct VTile {
    static constexpr int SW = Dim<D>::NG * 64 / 4;         // dwords of scales
    static constexpr int NS = (SW + 63) / 64;
    uint32_t w[Dim<D>::VD];
    uint32_t s[NS];
};
template <int D>
__device__ __forceinline__ void load_v(VTile<D>& v, const uint8_t* t, int lane) {
    constexpr int NG = Dim<D>::NG, SW = VTile<D>::SW;
#pragma unroll
    for (int j = 0; j < Dim<D>::VD / 4; ++j) {
        const uint4 x = *(const uint4*)(t + NG * 1088 + j * 1024 + lane * 16);
        v.w[4 * j] = x.x;
        v.w[4 * j + 1] = x.y;
        v.w[4 * j + 2] = x.z;
        v.w[4 * j + 3] = x.w;
    }
#pragma unroll
    for (int j = 0; j < VTile<D>::NS; ++j) v.s[j] = j * 64 + lane < SW ? *(const uint32_t*)(t + NG * 2112 + (j * 64 + lane) * 4) : 0u;
}
// To the wave's region of LDS; its earlier reads there are done (LDS keeps a wave's order).
template <int D>
__device__ __forceinline__ void put_v(const VTile<D>& v, uint8_t* region, int lane) {
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < Dim<D>::VD / 4; ++j)
        *(uint4*)(region + j * 1024 + lane * 16) = uint4{v.w[4 * j], v.w[4 * j + 1], v.w[4 * j + 2], v.w[4 * j + 3]};
#pragma unroll
    for (int j = 0; j < VTile<D>::NS; ++j)
        if (j * 64 + lane < VTile<D>::SW) *(uint32_t*)(region + Dim<D>::kVBytes + (j * 64 + lane) * 4) = v.s[j];
    __builtin_amdgcn_wave_barrier();
}
// Scales of positions from `end` (a position of the tile) on become 0: bytes there are no values, and a
// NaN scale would pass a zero weight. Returns whether another scale of the lane's is NaN.
template <int D>
__device__ __forceinline__ bool clear_v(VTile<D>& v, int end, int lane) {
    bool nan = false;
#pragma unroll
    for (int j = 0; j < VTile<D>::NS; ++j) {
        const int x = (((j * 64 + lane) * 4) & 63) >> 2;   // byte 4x + y of a group: position 16 (x % 4) + 4 (x / 4) + y
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (16 * (x & 3) + 4 * (x >> 2) + y >= end) v.s[j] &= ~(255u << (8 * y));
            if (((v.s[j] >> (8 * y)) & 127u) == 127u) nan = true;
        }
    }
    return nan;
}

template <int D>
__device__ __forceinline__ void scores_of(const KTile<D>& k, const h16x8 (&qf)[Dim<D>::NW], f32x4 (&s)[4]) {
#pragma unroll
    for (int bl = 0; bl < 4; ++bl) {
        s[bl] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < Dim<D>::NW; ++w) s[bl] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_frag<D>(k, bl, w), qf[w], s[bl], 0, 0, 0);
    }
}

// A row's running maximum, sum and output.
template <int D>
struct Running {
    f32x4 o[Dim<D>::NH];
    float m, l;
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int h = 0; h < Dim<D>::NH; ++h) o[h] = f32x4{0.f, 0.f, 0.f, 0.f};
        m = -__builtin_inff();
        l = 0.0f;
    }
    // Exponentials of a tile's scores, rounded; what was summed is scaled to the new maximum.
    __device__ __forceinline__ void weigh(const f32x4 (&s)[4], float factor, h16x8 (&p)[2]) {
        float mx = s[0][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) mx = fmaxf(mx, s[e >> 2][e & 3]);
        mx = max_over_q(mx);
        if (__ballot(mx > m)) {
            const float nm = fmaxf(mx, m), safe = nm == -__builtin_inff() ? 0.0f : nm;
            const float alpha = __builtin_amdgcn_exp2f((m - safe) * factor);
            m = nm;
            l *= alpha;
#pragma unroll
            for (int h = 0; h < Dim<D>::NH; ++h) o[h] *= alpha;
        }
        const float top = m == -__builtin_inff() ? 0.0f : m;
        float add = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e >> 2][e & 3] - top, factor, kLift));
            add += x;
            p[e >> 3][e & 7] = (_Float16)x;
        }
        l += add;
    }
    // NaN scales in a tile that some row does not see whole leave it, and the rows that see such a position
    // (from lo to below hi, positions of the tile) get NaN in its group's columns.
    __device__ __forceinline__ void take_nan(uint8_t* region, int lo, int hi, int q) {
#pragma unroll
        for (int g = 0; g < Dim<D>::NG; ++g) {
            uint8_t* sb = region + Dim<D>::kVBytes + g * 64 + q * 16;
            uint32_t bad = 0;
            float hit = 0.0f;
#pragma unroll 1
            for (int e = 0; e < 16; ++e) {
                const int ps = 16 * (e >> 2) + 4 * q + (e & 3);
                if ((sb[e] & 127u) != 127u) continue;
                bad |= 1u << e;
                if (ps >= lo && ps < hi) hit = 1.0f;
            }
            const float add = max_over_q(hit) > 0.0f ? __builtin_nanf("") : 0.0f;
            o[2 * g] += add;
            o[2 * g + 1] += add;
            __builtin_amdgcn_wave_barrier();
#pragma unroll 1
            for (int e = 0; e < 16; ++e)
                if (bad >> e & 1u) sb[e] = 0;
        }
        __builtin_amdgcn_wave_barrier();
    }
    __device__ __forceinline__ void add_v(const uint8_t* region, const h16x8 (&p)[2], int c, int q) {
#pragma unroll
        for (int g = 0; g < Dim<D>::NG; ++g) {
            const uint4 sc = *(const uint4*)(region + Dim<D>::kVBytes + g * 64 + q * 16);
            const uint32_t sd[4] = {sc.x, sc.y, sc.z, sc.w};
            h16x2 sv[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sv[2 * e] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sd[e], 1.0f, false);
                sv[2 * e + 1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sd[e], 1.0f, true);
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int h = 2 * g + hh, pos = 16 * (c >> 2) + 4 * q + (c & 3);
                const i32x2 vt = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                    (__attribute__((address_space(3))) i32x2*)(region + h * 512 + pos * 8));
#pragma unroll
                for (int st = 0; st < 2; ++st)
                    o[h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        decode8((uint32_t)vt[st], sv[4 * st], sv[4 * st + 1], sv[4 * st + 2], sv[4 * st + 3]), p[st], o[h], 0, 0, 0);
            }
        }
    }
};

template <int D>
constexpr int wave_v_bytes() {
    return Dim<D>::kVBytes + Dim<D>::NG * 64;              // a wave's region: V codes and scales
}
template <int D>
constexpr int wave_join_bytes() {
    return Dim<D>::NH * 1024 + 128;                        // a wave's output, maxima and sums
}
// The waves of a workgroup meet in LDS, in order: each leaves its share, then takes every waves-th 16
// columns. each(h, output, maximum, sum) has columns 16 h + 4 q .. + 3 of row c.
template <int D, typename F>
__device__ __forceinline__ void join_waves(Running<D>& r, float factor, uint8_t* lds, int wave, int waves, const F& each) {
    constexpr int NH = Dim<D>::NH;
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    r.l = sum_over_q(r.l);
    __syncthreads();                                       // the regions are read
    f32x4* buf = (f32x4*)(lds + wave * wave_join_bytes<D>());
    float* ml = (float*)(buf + NH * 64);
#pragma unroll
    for (int h = 0; h < NH; ++h) buf[h * 64 + lane] = r.o[h];
    if (q == 0) {
        ml[c] = r.m;
        ml[16 + c] = r.l;
    }
    __syncthreads();
    for (int h = wave; h < NH; h += waves) {
        float jm = -__builtin_inff(), jl = 0.0f;
        for (int w = 0; w < waves; ++w) jm = fmaxf(jm, ((const float*)(lds + w * wave_join_bytes<D>() + NH * 1024))[c]);
        const float safe = jm == -__builtin_inff() ? 0.0f : jm;
        f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < waves; ++w) {
            const uint8_t* from = lds + w * wave_join_bytes<D>();
            const float* wml = (const float*)(from + NH * 1024) + c;
            const float f = __builtin_amdgcn_exp2f((wml[0] - safe) * factor);
            jl = __builtin_fmaf(wml[16], f, jl);
            acc += ((const f32x4*)from)[h * 64 + lane] * f;
        }
        each(h, acc, jm, jl);
    }
}

// A wave's tiles: entries first, first + step, ... below end of a list. look(i, place) says, per lane,
// which tile of 64 positions entry i names (below 0: none) and where it lies, so that 64 entries are
// looked up at once and no tile waits for a page number. hide(base, s, v) takes out what is not seen
// of the tile at position base, and says whether NaN values of v are left that some row must not meet;
// nan(base) then sees to them. A tile's bytes are asked for one tile ahead: K once its scores are
// formed, V once it is in LDS.
template <int D, typename Look, typename Hide, typename Nan>
__device__ __forceinline__ void walk_tiles(const uint8_t* cache, int first, int end, int step, const Look& look, const Hide& hide,
                                           const Nan& nan, const h16x8 (&qf)[Dim<D>::NW], float factor, Running<D>& r, uint8_t* region) {
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    KTile<D> k;
    VTile<D> v;
    for (; first < end; first += 64 * step) {
        const int i = first + lane * step;
        long long place = 0;
        const int tile = i < end ? look(i, place) : -1;
        uint64_t todo = __ballot(tile >= 0);
        if (!todo) continue;
        const int place_lo = (int)place, place_hi = (int)(place >> 32);
        const auto at = [&](int j) {
            return cache + ((long long)(uint32_t)__builtin_amdgcn_readlane(place_lo, j) |
                            (long long)__builtin_amdgcn_readlane(place_hi, j) << 32);
        };
        int j = __ffsll((unsigned long long)todo) - 1;
        {
            const uint8_t* t = at(j);
            load_k<D>(k, t, c, q);
            load_v<D>(v, t, lane);
        }
        while (todo) {
            todo &= todo - 1;
            const int base = __builtin_amdgcn_readlane(tile, j) << 6;
            j = todo ? __ffsll((unsigned long long)todo) - 1 : j;
            const uint8_t* next = at(j);
            f32x4 s[4];
            scores_of<D>(k, qf, s);
            if (todo) load_k<D>(k, next, c, q);
            const bool odd = hide(base, s, v);
            put_v<D>(v, region, lane);
            if (todo) load_v<D>(v, next, lane);
            h16x8 p[2];
            r.weigh(s, factor, p);
            if (odd) nan(base);
            r.add_v(region, p, c, q);
        }
    }
}

}  // namespace attn
}  // namespace xp
