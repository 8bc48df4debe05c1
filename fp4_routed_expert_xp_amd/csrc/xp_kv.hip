// xp_kv.hip — the 4-bit key/value cache: quantising rows into it, reading rows
// back, and evicting positions by accumulated attention weight.
#include "xp_kv_dev.h"

namespace xp {
namespace kv {

// Sequence of a row of a packed batch: the number of ends cu[1..B] at or below
// it (B for a row behind the last sequence). One wave, uniform row.
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ cu, int B, int row) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int b = 0; b < B; b += 64) {
        const bool in = b + lane < B && cu[b + lane + 1] <= row;
        const int c = __popcll(__ballot(in));
        n += c;
        if (c < 64) break;
    }
    return n;
}

template <int TYPE>
__device__ __forceinline__ void load8(const void* p, long long at, float v[8]) {
    if constexpr (TYPE == XP_F32) {
        const float4 a = *(const float4*)((const float*)p + at), b = *(const float4*)((const float*)p + at + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = *(const uint4*)((const uint16_t*)p + at);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == XP_BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                v[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] & 0xffff));
                v[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
            }
        }
    }
}

struct RowMap {
    const int32_t* cu;
    const int32_t* start;
    const int32_t* table;
    int batch;
    int rows;
};

// The row of this workgroup: its sequence's page-table row and position.
// false: the row belongs to no sequence. pos is -1 where the cache has no such position.
__device__ __forceinline__ bool place(const Geo& g, const RowMap& m, int row, const int32_t*& table_row, int& pos) {
    const int b = sequence_of(m.cu, m.batch, row);
    if (b >= m.batch) return false;
    const long long p = (long long)m.start[b] + row - m.cu[b];
    pos = p >= 0 && p < (long long)g.max_pages * g.page ? (int)p : -1;
    table_row = m.table + (long long)b * g.max_pages;
    return true;
}

// Quantise: a row's 2 * kv_heads * head_dim values as units of 8, one a thread;
// four neighbouring threads hold a group of 32 and share its scale (its largest
// magnitude over two quad swaps). Bound by bytes: 2 (or 4) a value in, 4.25 bits
// out. Each quad stores one chunk of 16 bytes of K or two of 8 of V; the lines
// that neighbouring positions share meet in L2.
template <int TYPE>
__global__ __launch_bounds__(256) void append_kernel(Geo g, RowMap m, const void* __restrict__ k, long long ks,
                                                     const void* __restrict__ v, long long vs, uint8_t* __restrict__ cache) {
    const int row = blockIdx.x;
    const int u = blockIdx.y * 256 + threadIdx.x;
    const int per = g.kv_heads * g.groups * 4;       // units of one row of k
    const int32_t* tr;
    int pos;
    if (!place(g, m, row, tr, pos) || pos < 0 || u >= 2 * per) return;   // per is a multiple of 8: quads stay whole
    const bool is_v = u >= per;
    const int w = is_v ? u - per : u;
    float x[8];
    load8<TYPE>(is_v ? v : k, (long long)row * (is_v ? vs : ks) + 8 * w, x);
    float amax = 0.0f;
    bool bad = false;                                 // fmax drops a NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        amax = fmaxf(amax, __builtin_fabsf(x[i]));
        bad |= !(__builtin_fabsf(x[i]) < __builtin_inff());
    }
    amax = bad ? __builtin_inff() : amax;
    amax = fmaxf(amax, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(amax), 0xB1, 0xF, 0xF, true)));
    amax = fmaxf(amax, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(amax), 0x4E, 0xF, 0xF, true)));
    const uint32_t sb = scale_byte(amax);
    const float s = e4m3_value(sb);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) codes |= e2m1_code(x[i], s) << (4 * i);
    const int head = w / (g.groups * 4), gi = (w >> 2) % g.groups, part = w & 3;
    const long long tile = tile_at(g, tr, head, pos);
    if (tile < 0) return;
    uint8_t* t = cache + tile;
    const int p = pos & 63;
    if (is_v) {
        *(uint32_t*)(t + v_code(g.groups, p, 2 * gi + (part >> 1)) + 4 * (part & 1)) = codes;
        if (part == 0) t[v_scale(g.groups, p, gi)] = (uint8_t)sb;
    } else {
        *(uint32_t*)(t + k_code(g.groups, p, gi) + 4 * part) = codes;
        if (part == 0) t[k_scale(g.groups, p, gi)] = (uint8_t)sb;
    }
}

// The reverse, exact in all three types: e2m1 times E4M3 has six significant
// bits and lies within 2^-10 .. 2688. Positions the cache does not have read 0.
template <int TYPE>
__global__ __launch_bounds__(256) void read_kernel(Geo g, RowMap m, const uint8_t* __restrict__ cache, void* __restrict__ k,
                                                   long long ks, void* __restrict__ v, long long vs) {
    typedef float f32x2v __attribute__((ext_vector_type(2)));
    const int row = blockIdx.x;
    const int u = blockIdx.y * 256 + threadIdx.x;
    const int per = g.kv_heads * g.groups * 4;
    const int32_t* tr;
    int pos;
    if (!place(g, m, row, tr, pos) || u >= 2 * per) return;
    const bool is_v = u >= per;
    const int w = is_v ? u - per : u;
    const int head = w / (g.groups * 4), gi = (w >> 2) % g.groups, part = w & 3;
    const long long tile = pos < 0 ? -1 : tile_at(g, tr, head, pos);
    uint32_t codes = 0;
    float s = 0.0f;
    if (tile >= 0) {
        const uint8_t* t = cache + tile;
        const int p = pos & 63;
        codes = *(const uint32_t*)(t + (is_v ? v_code(g.groups, p, 2 * gi + (part >> 1)) + 4 * (part & 1)
                                             : k_code(g.groups, p, gi) + 4 * part));
        s = e4m3_value(t[is_v ? v_scale(g.groups, p, gi) : k_scale(g.groups, p, gi)]);
    }
    f32x2v x[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
                   __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3)};
    void* out = is_v ? v : k;
    const long long at = (long long)row * (is_v ? vs : ks) + 8 * w;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i].x *= s;
        x[i].y *= s;
        if constexpr (TYPE == XP_BF16)
            o[i] = (uint32_t)bf16_rne(x[i].x) | (uint32_t)bf16_rne(x[i].y) << 16;
        else if constexpr (TYPE == XP_F16)
            o[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[i].x) |
                   (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[i].y) << 16;
    }
    if constexpr (TYPE == XP_F32) {
        *(float4*)((float*)out + at) = float4{x[0].x, x[0].y, x[1].x, x[1].y};
        *(float4*)((float*)out + at + 4) = float4{x[2].x, x[2].y, x[3].x, x[3].y};
    } else {
        *(uint4*)((uint16_t*)out + at) = uint4{o[0], o[1], o[2], o[3]};
    }
}

// ------------------------------------------------------------------ eviction
constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;

// Weights in the order of selection as unsigned keys: larger first, -0 as +0,
// NaN below every number.
__device__ __forceinline__ uint32_t weight_key(float w) {
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
    if (u == 0x80000000u) u = 0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One workgroup per (sequence, kv head): the positions to keep, ascending. The
// key of the last one kept among the unprotected positions is found by four
// counting passes of eight bits (each wave counts into its own 256 bins); then
// each wave walks its own run of positions, once to count and once to write.
__global__ __launch_bounds__(kSelThreads) void evict_select_kernel(Geo g, const int32_t* __restrict__ lens,
                                                                   const float* weights, long long w_stride, int keep,
                                                                   int sinks, int recent, int32_t* kept,
                                                                   float* weights_out, long long wo_stride, int wo_len) {
    __shared__ uint32_t bins[kSelWaves][256];
    __shared__ uint32_t total[256];
    __shared__ int pick[2];                       // the chosen bin and how many are wanted inside it
    __shared__ int n_over[kSelWaves], n_tie[kSelWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const long long bh = (long long)blockIdx.y * g.kv_heads + blockIdx.x;
    const long long cap = (long long)g.max_pages * g.page;
    int n = lens[blockIdx.y];
    n = n < 0 ? 0 : (n > cap ? (int)cap : n);
    const float* w = weights + bh * w_stride;
    int32_t* out = kept + bh * keep;
    float* wo = weights_out + bh * wo_stride;
    const int m = n < keep ? n : keep;
    for (int i = m + tid; i < keep; i += kSelThreads) out[i] = -1;
    if (n <= keep) {
        for (int i = tid; i < n; i += kSelThreads) out[i] = i;
    } else {
        const int lo = sinks, hi = n - recent;
        int want = keep - sinks - recent;         // from [lo, hi), which holds more than that
        uint32_t key = 0, known = 0;              // the leading bits of the last kept key
        for (int shift = 24; want > 0 && shift >= 0; shift -= 8) {
            for (int i = lane; i < 256; i += 64) bins[wave][i] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += kSelThreads) {
                const uint32_t k = weight_key(w[i]);
                if ((k & known) == key) atomicAdd(&bins[wave][(k >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid < 256) {
                uint32_t s = 0;
                for (int j = 0; j < kSelWaves; ++j) s += bins[j][tid];
                total[tid] = s;
            }
            __syncthreads();
            if (wave == 0) {
                // lane holds bins 4*lane .. +3; `above`: counts of the bins over its own
                const uint32_t t0 = total[4 * lane], t1 = total[4 * lane + 1], t2 = total[4 * lane + 2],
                               t3 = total[4 * lane + 3];
                const int own = (int)(t0 + t1 + t2 + t3);
                const int upto = wave_incl_sum(own);
                int above = __builtin_amdgcn_readlane(upto, 63) - upto;
                const uint32_t t[4] = {t0, t1, t2, t3};
#pragma unroll
                for (int j = 3; j >= 0; --j) {
                    if (above < want && above + (int)t[j] >= want) {
                        pick[0] = 4 * lane + j;
                        pick[1] = want - above;
                    }
                    above += (int)t[j];
                }
            }
            __syncthreads();
            key |= (uint32_t)pick[0] << shift;
            known |= 255u << shift;
            want = pick[1];
            __syncthreads();
        }
        // want: how many of the positions that hold exactly `key` are kept, the lowest first
        const bool any = keep > sinks + recent;
        const int run = ((n + kSelThreads - 1) / kSelThreads) * 64;
        const int from = wave * run, to = from + run < n ? from + run : n;
        int over = 0, tie = 0;
        for (int i0 = from; i0 < to; i0 += 64) {
            const int i = i0 + lane;
            const bool in = i < to, held = in && (i < lo || i >= hi);
            const uint32_t k = in && !held ? weight_key(w[i]) : 0u;
            over += __popcll(__ballot(held || (any && in && !held && k > key)));
            tie += __popcll(__ballot(any && in && !held && k == key));
        }
        if (lane == 0) {
            n_over[wave] = over;
            n_tie[wave] = tie;
        }
        __syncthreads();
        int at = 0, ties = 0;                     // kept positions and ties before this wave's run
        for (int j = 0; j < wave; ++j) {
            const int left = want - ties;
            at += n_over[j] + (n_tie[j] < left ? n_tie[j] : left);
            ties = n_tie[j] < left ? ties + n_tie[j] : want;
        }
        const uint64_t below = lane ? ~0ull >> (64 - lane) : 0ull;
        for (int i0 = from; i0 < to; i0 += 64) {
            const int i = i0 + lane;
            const bool in = i < to, held = in && (i < lo || i >= hi);
            const uint32_t k = in && !held ? weight_key(w[i]) : 0u;
            const bool is_tie = any && in && !held && k == key;
            const uint64_t bt = __ballot(is_tie);
            const bool yes = held || (any && in && !held && k > key) || (is_tie && ties + __popcll(bt & below) < want);
            const uint64_t by = __ballot(yes);
            if (yes) out[at + __popcll(by & below)] = i;
            at += __popcll(by);
            ties += __popcll(bt);
        }
    }
    __syncthreads();   // kept[] of this (sequence, head) is written: move its weights
    // Ascending sources never lie before their targets, so a step's loads (all done at
    // the barrier) come before every store that could touch them, also in place.
    for (int i0 = 0; i0 < m; i0 += 8 * kSelThreads) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kSelThreads + tid;
            x[j] = i < m ? w[out[i]] : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kSelThreads + tid;
            if (i < m) wo[i] = x[j];
        }
    }
    const int end = n < wo_len ? n : wo_len;
    for (int i = m + tid; i < end; i += kSelThreads) wo[i] = 0.0f;
}

constexpr int kMoveThreads = 512;
constexpr int kMoveSteps = 4;

// One workgroup per (group of 32 values of k or v, kv head, sequence): its kept
// positions' codes and scale bytes, in order. As above a step's loads are done
// before its stores, and later steps read only behind them, so the destination
// pages may be the source's own. Bound by bytes (17 in and out a position) and,
// for few positions, by the chain kept -> page table -> bytes of each step.
__global__ __launch_bounds__(kMoveThreads) void evict_move_kernel(Geo src, Geo dst, const int32_t* lens,
                                                                  const int32_t* __restrict__ table,
                                                                  const int32_t* __restrict__ dst_table,
                                                                  const int32_t* __restrict__ kept, int keep, uint8_t* cache,
                                                                  int32_t* lens_out) {
    const int tid = threadIdx.x;
    const int head = blockIdx.y, b = blockIdx.z;
    const int groups = src.groups;
    const bool is_v = (int)blockIdx.x >= groups;
    const int gi = is_v ? blockIdx.x - groups : blockIdx.x;
    const long long cap = (long long)src.max_pages * src.page;
    int n = lens[b];
    n = n < 0 ? 0 : (n > cap ? (int)cap : n);
    const int m = n < keep ? n : keep;           // the same when lens_out, which may be lens, is written already
    if (blockIdx.x == 0 && head == 0 && tid == 0) lens_out[b] = m;
    const int32_t* list = kept + ((long long)b * src.kv_heads + head) * keep;
    const int32_t* tr = table + (long long)b * src.max_pages;
    const int32_t* dr = dst_table + (long long)b * dst.max_pages;
    for (int i0 = 0; i0 < m; i0 += kMoveSteps * kMoveThreads) {
        uint4 c[kMoveSteps];
        uint8_t s[kMoveSteps];
        long long from[kMoveSteps];
        int p[kMoveSteps];
#pragma unroll
        for (int j = 0; j < kMoveSteps; ++j) {
            const int i = i0 + j * kMoveThreads + tid;
            const int at = i < m ? list[i] : 0;
            p[j] = at & 63;
            from[j] = i < m ? tile_at(src, tr, head, at) : -1;
        }
#pragma unroll
        for (int j = 0; j < kMoveSteps; ++j) {
            c[j] = uint4{0, 0, 0, 0};
            s[j] = 0;
            if (from[j] >= 0) {
                const uint8_t* t = cache + from[j];
                if (is_v) {
                    const uint2 a = *(const uint2*)(t + v_code(groups, p[j], 2 * gi));
                    const uint2 d = *(const uint2*)(t + v_code(groups, p[j], 2 * gi + 1));
                    c[j] = uint4{a.x, a.y, d.x, d.y};
                    s[j] = t[v_scale(groups, p[j], gi)];
                } else {
                    c[j] = *(const uint4*)(t + k_code(groups, p[j], gi));
                    s[j] = t[k_scale(groups, p[j], gi)];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kMoveSteps; ++j) {
            const int i = i0 + j * kMoveThreads + tid;
            if (i >= m) continue;
            const long long to = tile_at(dst, dr, head, i);
            if (to < 0) continue;
            uint8_t* t = cache + to;
            const int q = i & 63;
            if (is_v) {
                *(uint2*)(t + v_code(groups, q, 2 * gi)) = uint2{c[j].x, c[j].y};
                *(uint2*)(t + v_code(groups, q, 2 * gi + 1)) = uint2{c[j].z, c[j].w};
                t[v_scale(groups, q, gi)] = s[j];
            } else {
                *(uint4*)(t + k_code(groups, q, gi)) = c[j];
                t[k_scale(groups, q, gi)] = s[j];
            }
        }
    }
}

}  // namespace kv
}  // namespace xp

using namespace xp;
using namespace xp::kv;

XP_API size_t xp_kv_bytes(const xp_kv_dims* dims) {
    if (!dims || !geo_ok(dims)) return 0;
    return (size_t)dims->n_pages * dims->kv_heads * (dims->page / kTilePos) * tile_bytes(dims->head_dim / 32);
}

// Checks shared by append and read; XP_OK with rows or batch 0 means nothing to do.
static int check_rows(const xp_kv_dims* dims, int32_t batch, int32_t max_pages, int32_t rows, int32_t type, const void* k,
                      int64_t ks, const void* v, int64_t vs, const void* cu, const void* start, const void* table,
                      const void* cache) {
    const int st = check_geo(dims, batch, max_pages);
    if (st != XP_OK) return st;
    if (rows < 0 || type < XP_BF16 || type > XP_F32) return XP_ERR_SHAPE;
    if (rows == 0 || batch == 0) return XP_OK;
    if (!k || !v || !cu || !start || !table || !cache) return XP_ERR_NULL;
    const int64_t width = (int64_t)dims->kv_heads * dims->head_dim, unit = type == XP_F32 ? 4 : 8;
    if (ks < width || vs < width || ks % unit || vs % unit) return XP_ERR_SHAPE;
    if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(cache, 16) || !aligned_to(cu, 4) || !aligned_to(start, 4) ||
        !aligned_to(table, 4))
        return XP_ERR_SHAPE;
    return XP_OK;
}

XP_API int xp_kv_append(const xp_kv_dims* dims, int32_t batch, int32_t max_pages, int32_t rows, int32_t type, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, const int32_t* cu_rows, const int32_t* start,
                        const int32_t* table, uint8_t* cache, void* stream) {
    const int st = check_rows(dims, batch, max_pages, rows, type, k, k_stride, v, v_stride, cu_rows, start, table, cache);
    if (st != XP_OK) return st;
    if (rows == 0 || batch == 0) return XP_OK;
    const Geo g = geo_of(dims, max_pages);
    const RowMap m{cu_rows, start, table, batch, rows};
    const dim3 grid((unsigned)rows, (unsigned)((2 * g.kv_heads * g.groups * 4 + 255) / 256));
    hipStream_t s = (hipStream_t)stream;
    if (type == XP_BF16)
        hipLaunchKernelGGL(append_kernel<XP_BF16>, grid, dim3(256), 0, s, g, m, k, k_stride, v, v_stride, cache);
    else if (type == XP_F16)
        hipLaunchKernelGGL(append_kernel<XP_F16>, grid, dim3(256), 0, s, g, m, k, k_stride, v, v_stride, cache);
    else
        hipLaunchKernelGGL(append_kernel<XP_F32>, grid, dim3(256), 0, s, g, m, k, k_stride, v, v_stride, cache);
    return launch_status();
}

XP_API int xp_kv_read(const xp_kv_dims* dims, int32_t batch, int32_t max_pages, int32_t rows, int32_t type,
                      const int32_t* cu_rows, const int32_t* start, const int32_t* table, const uint8_t* cache, void* k,
                      int64_t k_stride, void* v, int64_t v_stride, void* stream) {
    const int st = check_rows(dims, batch, max_pages, rows, type, k, k_stride, v, v_stride, cu_rows, start, table, cache);
    if (st != XP_OK) return st;
    if (rows == 0 || batch == 0) return XP_OK;
    const Geo g = geo_of(dims, max_pages);
    const RowMap m{cu_rows, start, table, batch, rows};
    const dim3 grid((unsigned)rows, (unsigned)((2 * g.kv_heads * g.groups * 4 + 255) / 256));
    hipStream_t s = (hipStream_t)stream;
    if (type == XP_BF16)
        hipLaunchKernelGGL(read_kernel<XP_BF16>, grid, dim3(256), 0, s, g, m, cache, k, k_stride, v, v_stride);
    else if (type == XP_F16)
        hipLaunchKernelGGL(read_kernel<XP_F16>, grid, dim3(256), 0, s, g, m, cache, k, k_stride, v, v_stride);
    else
        hipLaunchKernelGGL(read_kernel<XP_F32>, grid, dim3(256), 0, s, g, m, cache, k, k_stride, v, v_stride);
    return launch_status();
}

XP_API int xp_kv_evict(const xp_kv_dims* dims, int32_t batch, int32_t max_pages, uint8_t* cache, const int32_t* table,
                       const int32_t* lens, const float* weights, int64_t w_stride, int32_t keep, int32_t sinks,
                       int32_t recent, int32_t dst_pages, const int32_t* dst_table, int32_t* kept, int32_t* lens_out,
                       float* weights_out, int64_t wo_stride, void* stream) {
    const int st = check_geo(dims, batch, max_pages);
    if (st != XP_OK) return st;
    if (check_geo(dims, batch, dst_pages) != XP_OK || keep < 1 || sinks < 0 || recent < 0 ||
        (int64_t)sinks + recent > keep || keep > (int64_t)dst_pages * dims->page)
        return XP_ERR_SHAPE;
    if (batch == 0) return XP_OK;
    if (!cache || !table || !lens || !weights || !dst_table || !kept || !lens_out || !weights_out) return XP_ERR_NULL;
    if (w_stride < (int64_t)max_pages * dims->page || wo_stride < keep || !aligned_to(cache, 16) || !aligned_to(table, 4) ||
        !aligned_to(lens, 4) || !aligned_to(weights, 4) || !aligned_to(dst_table, 4) || !aligned_to(kept, 4) ||
        !aligned_to(lens_out, 4) || !aligned_to(weights_out, 4))
        return XP_ERR_SHAPE;
    if (weights_out == weights && wo_stride != w_stride) return XP_ERR_SHAPE;   // rows would overlap others' sources
    const Geo g = geo_of(dims, max_pages), d = geo_of(dims, dst_pages);
    hipStream_t s = (hipStream_t)stream;
    const int wo_len = wo_stride > 0x7fffffff ? 0x7fffffff : (int)wo_stride;
    hipLaunchKernelGGL(evict_select_kernel, dim3(g.kv_heads, batch), dim3(kSelThreads), 0, s, g, lens, weights,
                       (long long)w_stride, keep, sinks, recent, kept, weights_out, (long long)wo_stride, wo_len);
    const int rc = launch_status();
    if (rc != XP_OK) return rc;
    hipLaunchKernelGGL(evict_move_kernel, dim3(2 * g.groups, g.kv_heads, batch), dim3(kMoveThreads), 0, s, g, d, lens, table,
                       dst_table, kept, keep, cache, lens_out);
    return launch_status();
}
