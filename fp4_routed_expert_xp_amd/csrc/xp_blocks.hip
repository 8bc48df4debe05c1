// xp_blocks.hip — summaries of the cache's blocks of 64 positions, and the choice of the
// blocks that a query row attends to by a cheap score over them.
//
// Everything here is whole numbers, so the chosen lists are a function of the inputs
// alone, whatever the order of sums:
//  - a cached key is e2m1 (halves, up to 6) times E4M3 (multiples of 2^-9, up to 448): a
//    whole number of 2^-10, below 2^22; 64 of them add up to less than 2^28;
//  - a block's summary is that sum by 2^k in whole steps, head_dim signed bytes;
//  - a row's q is held as signed bytes by head, times a power of two;
//  - the product of both is below 127 * 127 * 256 < 2^22, exact in the matrix cores' int32
//    and in fp32, where the powers of two follow.
#include "xp_kv_dev.h"

namespace xp {
namespace blocks {

using kv::Geo;

typedef int i32x4 __attribute__((ext_vector_type(4)));

// The summaries' buffer: head_dim bytes of every entry, then a byte k of every entry;
// entries are [n_pages][kv_heads][page / 64], as the cache's tiles are.
__host__ __device__ __forceinline__ long long entries_of(const Geo& g) {
    return (long long)g.n_pages * g.kv_heads * (g.page / kv::kTilePos);
}

struct Rows {
    const int32_t* cu;
    const int32_t* start;
    const int32_t* table;
    int batch, rows;
};

// The sequence of this lane's row, rows of a wave being consecutive from `first` on.
__device__ __forceinline__ int lane_sequence(const Rows& m, int first) {
    const int lane = threadIdx.x & 63, row = first + lane;
    if (m.batch <= 64) {
        const int end = lane < m.batch ? m.cu[lane + 1] : 0x7fffffff;
        int n = 0;
        for (int b = 0; b < m.batch; ++b) n += __builtin_amdgcn_readlane(end, b) <= row;
        return n;
    }
    int lo = kv::sequence_of_row(m.cu, m.batch, first), hi = kv::sequence_of_row(m.cu, m.batch, first + 63);
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (m.cu[mid + 1] > row)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Lanes on either side of a pair keep a or b, and add the other side's.
template <int CTRL>
__device__ __forceinline__ int halve(int a, int b, bool up) {
    const int give = up ? a : b, own = up ? b : a;
    return own + __builtin_amdgcn_mov_dpp(give, CTRL, 0xf, 0xf, true);
}

// Bound by its chain of three loads for a step (32 sequences of 16 rows: 7 us), and by the reads
// of complete blocks for prompts (six of up to 8,100 rows: 18 MB in 12 us, in runs of a kilobyte).
// One workgroup: 64 rows and a kv head; a wave for each group of 32 values. The rows at a
// block's last position complete it: most often one of 64 consecutive rows. A wave takes a
// position a lane (16 bytes of codes and their scale), and halves values and lanes
// together, so that 32 sums over 64 lanes cost 32 exchanges of one instruction.
template <int NG>
__global__ __launch_bounds__(64 * NG) void blocks_kernel(Geo g, Rows m, const uint8_t* __restrict__ cache,
                                                         uint8_t* __restrict__ out) {
    __shared__ uint32_t tops[2][NG];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int first = (int)(blockIdx.x / g.kv_heads) * 64, head = blockIdx.x % g.kv_heads;
    const int b = lane_sequence(m, first);
    long long tile = -1;
    if (first + lane < m.rows && b < m.batch) {
        const long long at = (long long)m.start[b] + (first + lane - m.cu[b]);
        if ((at & 63) == 63 && at >= 0 && at < (long long)g.max_pages * g.page) {
            const int col = (int)at / g.page, id = m.table[(long long)b * g.max_pages + col];
            if ((unsigned)id < (unsigned)g.n_pages)
                tile = ((long long)id * g.kv_heads + head) * (g.page / kv::kTilePos) + ((int)at - col * g.page) / kv::kTilePos;
        }
    }
    uint64_t todo = __ballot(tile >= 0);
    const int tile_lo = (int)tile, tile_hi = (int)(tile >> 32);
    for (int turn = 0; todo; todo &= todo - 1, turn ^= 1) {
        const int l = __ffsll((unsigned long long)todo) - 1;
        const long long entry = (long long)(uint32_t)__builtin_amdgcn_readlane(tile_lo, l) |
                                (long long)__builtin_amdgcn_readlane(tile_hi, l) << 32;
        const uint8_t* t = cache + entry * kv::tile_bytes(NG);
        const uint4 c = *(const uint4*)(t + wave * 1024 + lane * 16);
        const uint32_t sb = t[kv::k_scale(NG, lane, wave)];
        // in units of 2^-10; a NaN scale's values count as zeros
        const float s = (sb & 127u) == 127u ? 0.0f : kv::e4m3_value(sb) * 1024.0f;
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        int v[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 1);
            const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 3);
            v[8 * i] = (int)(p0.x * s);
            v[8 * i + 1] = (int)(p0.y * s);
            v[8 * i + 2] = (int)(p1.x * s);
            v[8 * i + 3] = (int)(p1.y * s);
            v[8 * i + 4] = (int)(p2.x * s);
            v[8 * i + 5] = (int)(p2.y * s);
            v[8 * i + 6] = (int)(p3.x * s);
            v[8 * i + 7] = (int)(p3.y * s);
        }
        // halves of the lanes swap halves of the values and add: lane l ends with the sum of value l / 2
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const auto x = __builtin_amdgcn_permlane32_swap(v[i], v[i + 16], false, false);
            v[i] = (int)(x[0] + x[1]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const auto x = __builtin_amdgcn_permlane16_swap(v[i], v[i + 8], false, false);
            v[i] = (int)(x[0] + x[1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = halve<0x128>(v[i], v[i + 4], lane & 8);   // row_ror:8
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = halve<0x141>(v[i], v[i + 2], lane & 4);   // row_half_mirror
        v[0] = halve<0x4e>(v[0], v[1], lane & 2);                                    // quad_perm 2,3,0,1
        const int total = v[0] + __builtin_amdgcn_mov_dpp(v[0], 0xb1, 0xf, 0xf, true);   // quad_perm 1,0,3,2
        const uint32_t mag = (uint32_t)(total < 0 ? -total : total);
        const uint32_t top = wave_max_u32(mag);
        if (lane == 0) tops[turn][wave] = top;
        __syncthreads();
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < NG; ++i) most = tops[turn][i] > most ? tops[turn][i] : most;
        // the smallest k with most <= 127 * 2^k
        int k = 0;
        if (most > 127u) {
            k = 25 - __builtin_clz(most);      // most in [2^(k + 6), 2^(k + 7))
            k += most > 127u << k;
        }
        // whole steps of 2^k, ties to even; below 2^28, so nothing overflows
        const uint32_t half = k ? (1u << (k - 1)) - 1u + ((mag >> k) & 1u) : 0u;
        const int code = (int)((mag + half) >> k);
        if ((lane & 1) == 0) out[entry * (32 * NG) + wave * 32 + (lane >> 1)] = (uint8_t)(total < 0 ? -code : code);
        if (lane == 0 && wave == 0) out[entries_of(g) * (32 * NG) + entry] = (uint8_t)k;
    }
}

// ------------------------------------------------------------------ selection
constexpr int kMaxBlocks = 16384;   // of a sequence: their keys are held in LDS
constexpr int kShort = 2048;        // up to so many a wave holds in registers
constexpr int kSpare = 8;           // lanes more than are kept that end the search for a bound
constexpr int kCus = 256;

struct Select {
    Geo g;
    Rows m;
    const void* q;
    long long q_stride;
    const uint8_t* codes;
    const uint8_t* exps;
    int32_t* sel;
    int group, keep, sinks, recent;
    int together;         // rows of a workgroup
};

// A score as an unsigned key in the same order; 0 is below all of them.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float max_over_q(float x) {
    uint32_t u = __float_as_uint(x);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    u = __float_as_uint(x);
    auto b = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// q of 16 heads as the matrix cores' operand: lane (c, p) holds the head at `from` at dims
// 64 st + 16 p .. + 15. Returns the exponent e of its steps, the smallest with |q| <= 127 * 2^e;
// a head that is zero, not finite or not there has zeros and kNone.
constexpr int kNone = -1000;
template <int D, bool BF16>
__device__ __forceinline__ int quantise_q(const uint16_t* from, bool there, i32x4 (&code)[D / 64]) {
    const int p = (threadIdx.x & 63) >> 4;
    float x[D / 64][16], top = 0.0f;
    bool odd = false;
#pragma unroll
    for (int st = 0; st < D / 64; ++st) {
        const uint4 u0 = *(const uint4*)(from + 64 * st + 16 * p), u1 = *(const uint4*)(from + 64 * st + 16 * p + 8);
        const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (BF16) {
                x[st][2 * i] = __uint_as_float(w[i] << 16);
                x[st][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                x[st][2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] & 0xffff));
                x[st][2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float m = __builtin_fabsf(x[st][i]);
            odd |= !(m < __builtin_inff());
            top = fmaxf(top, m);
        }
    }
    top = max_over_q(odd ? __builtin_inff() : top);
    int e = kNone;
    if (there && top > 0.0f && top < __builtin_inff()) {
        e = __builtin_amdgcn_frexp_expf(top) - 7;
        e += __builtin_amdgcn_frexp_mantf(top) > 127.0f / 128.0f;
    }
#pragma unroll
    for (int st = 0; st < D / 64; ++st)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float y = __builtin_rintf(__builtin_amdgcn_ldexpf(x[st][4 * j + i], e == kNone ? 0 : -e));
                w |= (e == kNone ? 0u : (uint32_t)(int)y & 255u) << (8 * i);
            }
            code[st][j] = (int)w;
        }
    return e;
}

// One step's shared part of both kernels below: the keys of the blocks [0, n) of T rows of one
// sequence and a kv head into keys[T][pitch]. A wave takes 64 blocks: a lane looks up one
// block's page, four products of 16 blocks by 16 (row, head) pairs follow, and a lane ends with
// its own block's scores. Blocks without a page get the key 1, below that of any score.
template <int D, bool BF16, int T>
__device__ __forceinline__ void score_blocks(const Select& a, int row, int rows, int head, int b, int n, uint32_t* keys, int pitch) {
    const int lane = threadIdx.x & 63, c = lane & 15, p = lane >> 4, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t* table = a.m.table + (long long)b * a.g.max_pages;
    const int tiles = a.g.page / kv::kTilePos;
    // pair c of a sixteen from h0 on: row t and head h; T > 1 takes all heads at once
    const int t = T > 1 ? c / a.group : 0, h = T > 1 ? c - t * a.group : c;
    const auto at = [&](int h0) {
        const bool there = t < rows && h0 + h < a.group && t < T;
        return there ? (const uint16_t*)a.q + (long long)(row + t) * a.q_stride + ((long long)head * a.group + h0 + h) * D : nullptr;
    };
    const uint16_t* any = (const uint16_t*)a.q + (long long)row * a.q_stride + (long long)head * a.group * D;
    // a lane's block of the wave's next 64, and its page: asked for ahead
    const auto look = [&](int base) { return table[(base + lane < n ? base + lane : n - 1) / tiles]; };
    int id = wave * 64 < n ? look(wave * 64) : -1;
    i32x4 code[D / 64];
    int e = quantise_q<D, BF16>(at(0) ? at(0) : any, at(0), code), top = e;
    if (T == 1)
        for (int h0 = 16; h0 < a.group; h0 += 16) {
            i32x4 unused[D / 64];
            const int other = quantise_q<D, BF16>(at(h0) ? at(h0) : any, at(h0), unused);
            top = other > top ? other : top;
        }
    for (int i = 1; i < (T > 1 ? a.group : 16); i <<= 1) {
        const int other = __shfl_xor(top, i);
        top = other > top ? other : top;
    }
    for (int h0 = 0; h0 < a.group; h0 += 16) {
        if (h0) e = quantise_q<D, BF16>(at(h0) ? at(h0) : any, at(h0), code);
        // each head's steps against the largest ones', down to 2^-64 of them
        const float f = __builtin_amdgcn_ldexpf(1.0f, e - top < -64 ? -64 : e - top);
        float fr[4];
        int of[4];                             // whose row the lane's four results are
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fr[i] = __shfl(f, 4 * p + i);
            of[i] = T > 1 ? (4 * p + i) / a.group : (h0 + 4 * p + i < a.group ? 0 : -1);
        }
        for (int base = wave * 64; base < n; base += waves * 64) {
            const int blk = base + lane < n ? base + lane : n - 1, col = blk / tiles;
            const bool there = (unsigned)id < (unsigned)a.g.n_pages;
            const long long entry = there ? ((long long)id * a.g.kv_heads + head) * tiles + (blk - col * tiles) : 0;
            const int k = a.exps[entry], next = base + waves * 64;
            if (next < n || h0 + 16 < a.group) id = look(next < n ? next : wave * 64);
            i32x4 m[4][D / 64];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const long long from = (long long)(uint32_t)__shfl((int)entry, 16 * u + c) | (long long)__shfl((int)(entry >> 32), 16 * u + c) << 32;
#pragma unroll
                for (int st = 0; st < D / 64; ++st) m[u][st] = *(const i32x4*)(a.codes + from * D + 64 * st + 16 * p);
            }
            if (T > 1 && a.group == 4) {       // a lane's four results are one row's: it keeps those
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    i32x4 acc = i32x4{0, 0, 0, 0};
#pragma unroll
                    for (int st = 0; st < D / 64; ++st) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(code[st], m[u][st], acc, 0, 0, 0);
                    const float most = fmaxf(fmaxf((float)acc[0] * fr[0], (float)acc[1] * fr[1]), fmaxf((float)acc[2] * fr[2], (float)acc[3] * fr[3]));
                    const int at = 16 * u + c, ku = __shfl(there ? k : -1, at);
                    if (p < rows && base + at < n) keys[p * pitch + base + at] = ku < 0 ? 1u : key_of(__builtin_amdgcn_ldexpf(most, ku));
                }
                continue;
            }
            float best[T];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                i32x4 acc = i32x4{0, 0, 0, 0};
#pragma unroll
                for (int st = 0; st < D / 64; ++st) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(code[st], m[u][st], acc, 0, 0, 0);
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = (float)acc[i] * fr[i];
#pragma unroll
                for (int r = 0; r < T; ++r) {
                    float most = -__builtin_inff();
#pragma unroll
                    for (int i = 0; i < 4; ++i) most = fmaxf(most, of[i] == r ? x[i] : -__builtin_inff());
                    most = max_over_q(most);
                    best[r] = u == 0 || p == u ? most : best[r];
                }
            }
            if (base + lane < n)
#pragma unroll
                for (int r = 0; r < T; ++r) {
                    if (r >= rows) break;
                    const uint32_t key = there ? key_of(__builtin_amdgcn_ldexpf(best[r], k)) : 1u;
                    uint32_t* to = keys + r * pitch + blk;
                    *to = h0 && *to > key ? *to : key;
                }
        }
    }
}

// Blocks up to a row's own.
__device__ __forceinline__ int blocks_of(const Select& a, int row, int b) {
    const int cap = a.g.max_pages * a.g.page;
    long long pos = (long long)a.m.start[b] + (row - a.m.cu[b]);
    pos = pos >= cap ? cap - 1 : pos;
    return pos < 0 ? 0 : (int)(pos >> 6) + 1;
}

// A wave lists the blocks of one row from their keys, in registers: the key of the last one
// kept is the largest T with as many keys at or above it as are kept, found bit by bit; once
// there are just as many the rest of its bits does not matter.
// Up to 64 kept, few lanes' largest keys tell which keys are worth it: as many lanes as are kept have
// one at or above some bound, so the last one kept is not below it. What is at or above it is most often
// a wave's worth, a key a lane, in `few` (512 rows of 16 blocks of 1,016: 31.2 us without, 26.5 with).
struct Few {
    uint32_t key;
    int block;
};
template <int KPL>
__device__ __forceinline__ void list_blocks(const Select& a, const uint32_t* keys, int n, int32_t* out, Few* few) {
    const int lane = threadIdx.x & 63, last = n - a.recent;
    uint32_t k[KPL], top = 0;                  // top: of those that are not listed anyway
#pragma unroll
    for (int j = 0; j < KPL; ++j) {
        const int i = j * 64 + lane;
        const bool open = i >= a.sinks && i < last;
        k[j] = i >= n ? 0u : (open ? keys[i] : ~0u);
        top = open && k[j] > top ? k[j] : top;
    }
    top = wave_max_u32(top);
    const uint64_t below = (1ull << lane) - 1;
    if (a.keep <= 64) {
        uint32_t own = k[0], bound = 0;
#pragma unroll
        for (int j = 1; j < KPL; ++j) own = k[j] > own ? k[j] : own;
#pragma unroll 1
        for (int bit = 31; bit >= 0; --bit) {
            const int lanes = __popcll(__ballot(own >= (bound | 1u << bit)));
            if (lanes < a.keep) continue;
            bound |= 1u << bit;
            if (lanes <= a.keep + kSpare) break;
        }
        int held = 0;
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
            const uint64_t in = __ballot(k[j] >= bound);
            const int to = held + __popcll(in & below);
            if (k[j] >= bound && to < 64) few[to] = Few{k[j], j * 64 + lane};
            held += __popcll(in);
        }
        if (held <= 64) {
            __builtin_amdgcn_wave_barrier();
            const Few x = lane < held ? few[lane] : Few{0u, 0};
            uint32_t key = 0;
            int count = held;                  // at or above `key`
#pragma unroll 1
            for (int bit = 31; bit >= 0 && count != a.keep; --bit) {
                const int lanes = __popcll(__ballot(x.key >= (key | 1u << bit)));
                if (lanes < a.keep) continue;
                key |= 1u << bit;
                count = lanes;
            }
            const uint64_t same = __ballot(x.key == key && lane < held);
            const int ties = a.keep - __popcll(__ballot(x.key > key));
            const bool yes = lane < held && (x.key > key || (x.key == key && __popcll(same & below) < ties));
            const uint64_t chosen = __ballot(yes);
            if (yes) out[__popcll(chosen & below)] = x.block;
            return;
        }
    }
    uint32_t key = 0;
    int over = 0, count = 0;                   // keys above `key`; at or above what is tried
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t t = key | 1u << bit;
        if (t > top) continue;                 // less than are kept: some of them are open
        count = 0;
#pragma unroll
        for (int j = 0; j < KPL; ++j) count += k[j] >= t;
        count = __builtin_amdgcn_readlane(wave_incl_sum(count), 63);
        if (count >= a.keep) key = t;
        if (count == a.keep) break;
    }
    int ties = 0;                              // of the keys equal to `key`: the lowest blocks
    if (count != a.keep) {
#pragma unroll
        for (int j = 0; j < KPL; ++j) over += k[j] > key;
        ties = a.keep - __builtin_amdgcn_readlane(wave_incl_sum(over), 63);
    } else {
        ties = a.keep;                         // more than there are: all of them
    }
    int at = 0;
#pragma unroll
    for (int j = 0; j < KPL; ++j) {
        const uint64_t same = __ballot(k[j] == key);
        const bool yes = k[j] > key || (k[j] == key && __popcll(same & below) < ties);
        const uint64_t chosen = __ballot(yes);
        if (yes) out[at + __popcll(chosen & below)] = j * 64 + lane;
        at += __popcll(chosen);
        ties -= __popcll(same);
        ties = ties < 0 ? 0 : ties;
    }
}

// Four rows (two of eight heads) and a kv head a workgroup, up to kShort blocks: scores by all
// waves, lists by a wave each. Rows of one sequence share the summaries they read and the
// products' 16 pairs.
template <int D, bool BF16>
__global__ __launch_bounds__(256, D == 256 ? 2 : 4) void select_kernel(Select a) {
    extern __shared__ uint32_t keys[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.x % a.g.kv_heads, pitch = a.g.max_pages * (a.g.page / kv::kTilePos);
    Few* few = (Few*)(keys + a.together * pitch) + 64 * wave;
    int row = (int)(blockIdx.x / a.g.kv_heads) * a.together;
    const int end = row + a.together < a.m.rows ? row + a.together : a.m.rows;
    while (row < end) {
        const int b = kv::sequence_of_row(a.m.cu, a.m.batch, row);
        if (b >= a.m.batch) return;            // rows behind the last sequence
        const int stop = a.m.cu[b + 1], next = stop > row && stop < end ? stop : end, rows = next - row;
        const int most = blocks_of(a, next - 1, b);        // the last row's are the most
        if (most > a.keep && a.keep > a.sinks + a.recent) score_blocks<D, BF16, 4>(a, row, rows, head, b, most, keys, pitch);
        __syncthreads();
        if (wave < rows) {
            const int n = blocks_of(a, row + wave, b);
            int32_t* out = a.sel + ((long long)(row + wave) * a.g.kv_heads + head) * a.keep;
            if (n <= a.keep)
                for (int i = lane; i < a.keep; i += 64) out[i] = i < n ? i : -1;
            else if (a.keep == a.sinks + a.recent)
                for (int i = lane; i < a.keep; i += 64) out[i] = i < a.sinks ? i : n - a.keep + i;
            else if (n <= 256)
                list_blocks<4>(a, keys + wave * pitch, n, out, few);
            else if (n <= 512)
                list_blocks<8>(a, keys + wave * pitch, n, out, few);
            else if (n <= 1024)
                list_blocks<16>(a, keys + wave * pitch, n, out, few);
            else
                list_blocks<kShort / 64>(a, keys + wave * pitch, n, out, few);
        }
        row = next;
        __syncthreads();
    }
}

// A row and a kv head a workgroup, any number of blocks: the key of the last block kept by
// counting passes of 8 bits over LDS; then each wave walks its run of blocks, once to count
// and once to write. (Rows alone through the kernel above, listed by one wave from registers, take
// 12.5 us where this takes 9.8: 30 rows of 8 kv heads over up to 516 blocks, in a graph. Over up to
// 1,564 they take 23.7 and 16.1; 10 rows over up to 316 10.8 and 8.2.)
template <int D, bool BF16>
__global__ __launch_bounds__(1024) void select_row_kernel(Select a) {
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t bins[256];
    __shared__ int pick[2];
    __shared__ int n_over[16], n_tie[16];
    const int tid = threadIdx.x, lane = tid & 63, threads = blockDim.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = (int)(blockIdx.x / a.g.kv_heads), head = blockIdx.x % a.g.kv_heads;
    const int b = kv::sequence_of_row(a.m.cu, a.m.batch, row);
    if (b >= a.m.batch) return;                // rows behind the last sequence
    int32_t* out = a.sel + ((long long)row * a.g.kv_heads + head) * a.keep;
    const int n = blocks_of(a, row, b), m = n < a.keep ? n : a.keep;
    for (int i = m + tid; i < a.keep; i += threads) out[i] = -1;
    if (n <= a.keep) {
        for (int i = tid; i < n; i += threads) out[i] = i;
        return;
    }
    const int lo = a.sinks, hi = n - a.recent;
    int want = a.keep - a.sinks - a.recent;    // of [lo, hi), which holds more than that
    uint32_t key = 0;
    if (want > 0) {
        score_blocks<D, BF16, 1>(a, row, 1, head, b, n, keys, 0);
        __syncthreads();
        uint32_t known = 0;
#pragma unroll 1
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += threads) bins[i] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += threads) {
                const uint32_t k = keys[i];
                if ((k & known) == key) atomicAdd(&bins[(k >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (wave == 0) {                   // lane l has bins 255 - 4 l - j: the largest first
                int own[4], sum = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    own[j] = (int)bins[255 - 4 * lane - j];
                    sum += own[j];
                }
                int above = wave_incl_sum(sum) - sum;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (above < want && above + own[j] >= want) {
                        pick[0] = 255 - 4 * lane - j;
                        pick[1] = want - above;
                    }
                    above += own[j];
                }
            }
            __syncthreads();
            key |= (uint32_t)pick[0] << shift;
            known |= 255u << shift;
            want = pick[1];
        }
    }
    // want: how many of the blocks that hold exactly `key` are kept, the lowest first
    const int run = (n + threads - 1) / threads * 64;
    const int from = wave * run, to = from + run < n ? from + run : n;
    const bool any = a.keep > a.sinks + a.recent;
    int over = 0, tie = 0;
    for (int i0 = from; i0 < to; i0 += 64) {
        const int i = i0 + lane;
        const bool in = i < to, held = in && (i < lo || i >= hi), open = any && in && !held;
        const uint32_t k = open ? keys[i] : 0u;
        over += __popcll(__ballot(held || (open && k > key)));
        tie += __popcll(__ballot(open && k == key));
    }
    if (lane == 0) {
        n_over[wave] = over;
        n_tie[wave] = tie;
    }
    __syncthreads();
    int at = 0, ties = 0;                      // kept blocks and ties before this wave's run
    for (int j = 0; j < wave; ++j) {
        const int left = want - ties;
        at += n_over[j] + (n_tie[j] < left ? n_tie[j] : left);
        ties = n_tie[j] < left ? ties + n_tie[j] : want;
    }
    const uint64_t below = lane ? ~0ull >> (64 - lane) : 0ull;
    for (int i0 = from; i0 < to; i0 += 64) {
        const int i = i0 + lane;
        const bool in = i < to, held = in && (i < lo || i >= hi), open = any && in && !held;
        const uint32_t k = open ? keys[i] : 0u;
        const bool is_tie = open && k == key;
        const uint64_t bt = __ballot(is_tie);
        const bool yes = held || (open && k > key) || (is_tie && ties + __popcll(bt & below) < want);
        const uint64_t by = __ballot(yes);
        if (yes) out[at + __popcll(by & below)] = i;
        at += __popcll(by);
        ties += __popcll(bt);
    }
}

static int check_rows(const xp_kv_dims* d, int32_t batch, int32_t max_pages, int32_t rows) {
    const int st = kv::check_geo(d, batch, max_pages);
    if (st != XP_OK) return st;
    // a workgroup for each kv head and row: a launch has fewer than 2^32 threads
    return rows < 0 || (int64_t)rows * d->kv_heads >= (1 << 22) ? XP_ERR_SHAPE : XP_OK;
}

template <int D, bool BF16>
static int launch(Select a, int most, hipStream_t s) {
    const long long pairs = (long long)a.m.rows * a.g.kv_heads;
    // Rows of a sequence share a workgroup where they are neighbours on average and there are more than
    // three for each CU, or one where blocks are many. 8 kv heads, us shared and one by one:
    //   4 heads of each: 47 blocks 64 rows 8.6 and 7.3, 128 rows 8.7 and 9.0, 256 rows 10.4 and 13.4; 316
    //   blocks 64 rows 11.1 and 10.7, 90 11.1 and 11.9, 128 11.3 and 13.2; 520 blocks 36 rows 12.7 and 11.8,
    //   64 12.8 and 13.0, 128 13.2 and 17.6; 816 blocks 36 rows 13.6 and 14.3, 64 13.9 and 16.0; 1,020 blocks
    //   36 rows 14.2 and 15.8, 128 14.7 and 24.7; 512 rows 27 and 68.
    // One, two and eight heads pay more for sharing, so that the rule takes the slower side for up to 64 rows
    // between 512 and 816 blocks and, of eight heads, for 90: 520 blocks 36 rows of two 14.3 and 11.9, 64 14.4
    // and 13.0, 90 14.7 and 15.2, 90 of eight 17.2 and 15.5; 816 blocks 36 rows of two 15.7 and 14.3, 64 16.2
    // and 15.8; 1,020 blocks 36 rows of two 16.0 and 15.7, of eight 15.9 and 15.9.
    // Groups of other sizes (3, 5, 6, 7, more than 8) are always one by one: 512 rows over 1,016 blocks take
    // 74 us of five and 71 of seven heads, 51 of eight. `most` is the table's: one of more than kShort
    // blocks has all rows one by one, and LDS for every block, however short its sequences are.
    const bool many = most <= kShort && (a.group == 1 || a.group == 2 || a.group == 4 || a.group == 8) &&
                      a.m.rows >= 4ll * a.m.batch && pairs > (most > 512 ? 1 : 3) * kCus;
    a.together = !many ? 1 : (a.group == 8 ? 2 : 4);
    const long long groups = ((long long)a.m.rows + a.together - 1) / a.together * a.g.kv_heads;
    // Waves take 64 blocks at a time: as many as there are such rounds, up to eight beyond a workgroup for
    // each CU, four from two on (8 kv heads, 940 blocks: 40 rows in fifteen waves 20 us, in eight 15.6, in
    // four 16.7; 100 rows in fifteen 34, in four 21).
    const int rounds = (most + 63) / 64, top = groups > kCus ? 8 : 16;
    const int waves = many || groups >= 2 * kCus || rounds < 4 ? 4 : (rounds < top ? rounds : top);
    const dim3 grid((unsigned)groups), block(64 * waves);
    const unsigned lds = (unsigned)most * 4 * a.together + (many ? 4 * 64 * sizeof(Few) : 0);
    if (many)
        hipLaunchKernelGGL((select_kernel<D, BF16>), grid, block, lds, s, a);
    else
        hipLaunchKernelGGL((select_row_kernel<D, BF16>), grid, block, lds, s, a);
    return launch_status();
}

}  // namespace blocks
}  // namespace xp

using namespace xp;
using namespace xp::blocks;

XP_API size_t xp_kv_blocks_bytes(const xp_kv_dims* dims) {
    if (!dims || !kv::geo_ok(dims)) return 0;
    return (size_t)entries_of(kv::geo_of(dims, 1)) * (size_t)(dims->head_dim + 1);
}

XP_API int xp_kv_blocks(const xp_kv_dims* dims, int32_t batch, int32_t max_pages, int32_t rows, const int32_t* cu_rows,
                        const int32_t* start, const int32_t* table, const uint8_t* cache, uint8_t* blocks, void* stream) {
    const int st = kv::check_geo(dims, batch, max_pages);
    if (st != XP_OK) return st;
    if (rows < 0 || ((int64_t)rows + 63) / 64 * dims->kv_heads >= (1 << 23)) return XP_ERR_SHAPE;   // fewer than 2^32 threads
    if (batch == 0 || rows == 0) return XP_OK;
    if (!cu_rows || !start || !table || !cache || !blocks) return XP_ERR_NULL;
    if (!kv::aligned_to(cu_rows, 4) || !kv::aligned_to(start, 4) || !kv::aligned_to(table, 4) || !kv::aligned_to(cache, 16) ||
        !kv::aligned_to(blocks, 16))
        return XP_ERR_SHAPE;
    const Geo g = kv::geo_of(dims, max_pages);
    const kv::Rows read[] = {kv::flat(cache, (int64_t)xp_kv_bytes(dims)), kv::flat(cu_rows, 4 * (int64_t)batch + 4),
                             kv::flat(start, 4 * (int64_t)batch), kv::flat(table, 4 * (int64_t)batch * max_pages)};
    if (kv::meets_any(kv::flat(blocks, (int64_t)xp_kv_blocks_bytes(dims)), read, 4)) return XP_ERR_SHAPE;
    const Rows m{cu_rows, start, table, batch, rows};
    hipStream_t s = (hipStream_t)stream;
    const dim3 grid((unsigned)((rows + 63) / 64 * (int64_t)dims->kv_heads));
    if (g.groups == 2)
        hipLaunchKernelGGL(blocks_kernel<2>, grid, dim3(128), 0, s, g, m, cache, blocks);
    else if (g.groups == 4)
        hipLaunchKernelGGL(blocks_kernel<4>, grid, dim3(256), 0, s, g, m, cache, blocks);
    else
        hipLaunchKernelGGL(blocks_kernel<8>, grid, dim3(512), 0, s, g, m, cache, blocks);
    return launch_status();
}

XP_API int xp_attn_select(const xp_kv_dims* dims, int32_t heads, int32_t batch, int32_t max_pages, int32_t rows, int32_t type,
                          const void* q, int64_t q_stride, const int32_t* cu_rows, const int32_t* start, const int32_t* table,
                          const uint8_t* blocks, int32_t keep, int32_t sinks, int32_t recent, int32_t* sel, void* stream) {
    const int st = check_rows(dims, batch, max_pages, rows);
    if (st != XP_OK) return st;
    const int64_t most = (int64_t)max_pages * (dims->page / kv::kTilePos);
    if (heads < 1 || heads > 65535 || heads % dims->kv_heads || (type != XP_BF16 && type != XP_F16) || most > kMaxBlocks ||
        sinks < 0 || recent < 1 || (int64_t)sinks + recent > keep || keep > kMaxBlocks)
        return XP_ERR_SHAPE;
    if (batch == 0 || rows == 0) return XP_OK;
    if (!q || !cu_rows || !start || !table || !blocks || !sel) return XP_ERR_NULL;
    const int64_t width = (int64_t)heads * dims->head_dim;
    if (q_stride < width || q_stride % 8 || !kv::aligned_to(q, 16) || !kv::aligned_to(cu_rows, 4) || !kv::aligned_to(start, 4) ||
        !kv::aligned_to(table, 4) || !kv::aligned_to(blocks, 16) || !kv::aligned_to(sel, 4))
        return XP_ERR_SHAPE;
    const kv::Rows read[] = {kv::Rows{q, rows, 2 * q_stride, 2 * width}, kv::flat(cu_rows, 4 * (int64_t)batch + 4),
                             kv::flat(start, 4 * (int64_t)batch), kv::flat(table, 4 * (int64_t)batch * max_pages),
                             kv::flat(blocks, (int64_t)xp_kv_blocks_bytes(dims))};
    if (kv::meets_any(kv::flat(sel, (int64_t)rows * dims->kv_heads * keep * 4), read, 5)) return XP_ERR_SHAPE;
    Select a{};
    a.g = kv::geo_of(dims, max_pages);
    a.m = Rows{cu_rows, start, table, batch, rows};
    a.q = q;
    a.q_stride = q_stride;
    a.codes = blocks;
    a.exps = blocks + entries_of(a.g) * dims->head_dim;
    a.sel = sel;
    a.group = heads / dims->kv_heads;
    a.keep = keep;
    a.sinks = sinks;
    a.recent = recent;
    hipStream_t s = (hipStream_t)stream;
    const bool bf = type == XP_BF16;
    switch (dims->head_dim) {
        case 64: return bf ? launch<64, true>(a, (int)most, s) : launch<64, false>(a, (int)most, s);
        case 128: return bf ? launch<128, true>(a, (int)most, s) : launch<128, false>(a, (int)most, s);
        default: return bf ? launch<256, true>(a, (int)most, s) : launch<256, false>(a, (int)most, s);
    }
}
