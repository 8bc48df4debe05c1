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

// Where a row's position lies: bytes of the cache to kv head 0's tile, -1 where the
// cache has no such position, -2 for a row of no sequence; and its place in the tile.
// b: the row's sequence or an earlier one.
__device__ __forceinline__ long long place(const Geo& g, const RowMap& m, int row, int b, int& pos) {
    pos = 0;
    if (row >= m.rows) return -2;
    while (b < m.batch && m.cu[b + 1] <= row) ++b;
    if (b >= m.batch) return -2;
    const long long at = (long long)m.start[b] + row - m.cu[b];
    if (at < 0 || at >= (long long)g.max_pages * g.page) return -1;
    pos = (int)at & 63;
    return tile_at(g, m.table + (long long)b * g.max_pages, 0, (int)at);
}
// Bytes between kv heads' tiles of one page.
__device__ __forceinline__ long long head_step(const Geo& g) { return (long long)(g.page / kTilePos) * tile_bytes(g.groups); }

// A unit is 8 values of one row of k or v: per = 4 * groups units of k for each kv head,
// as many of v. Where a unit lies in its tile:
struct Unit {
    int gi, part;   // group of 32 values, quarter of it
    bool is_v;
};
__device__ __forceinline__ int code_at(const Geo& g, const Unit& u, int pos) {
    return u.is_v ? v_code(g.groups, pos, 2 * u.gi + (u.part >> 1)) + 4 * (u.part & 1) : k_code(g.groups, pos, u.gi) + 4 * u.part;
}
__device__ __forceinline__ int scale_at(const Geo& g, const Unit& u, int pos) {
    return u.is_v ? v_scale(g.groups, pos, u.gi) : k_scale(g.groups, pos, u.gi);
}

// One unit into its tile. Four neighbouring lanes hold a group and share its scale.
__device__ __forceinline__ void quantise(const Geo& g, const Unit& u, const float x[8], uint8_t* tile, int pos) {
    // magnitudes compare as integers, a NaN above infinity above every number
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t a = __float_as_uint(x[j]) & 0x7fffffffu;
        top = a > top ? a : top;
    }
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, true);
    top = o > top ? o : top;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xF, 0xF, true);
    top = o > top ? o : top;
    const uint32_t sb = scale_byte(__uint_as_float(top));
    const float s = e4m3_value(sb);
    uint32_t codes;
    if (sb == 0x7fu) {                               // not finite: signed zeros under a NaN scale
        codes = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) codes |= __float_as_uint(x[j]) >> 31 << (4 * j + 3);
    } else {
        codes = e2m1_codes(x, s, s > 0.0f ? 1.0f / s : 0.0f);
    }
    *(uint32_t*)(tile + code_at(g, u, pos)) = codes;
    if (u.part == 0) tile[scale_at(g, u, pos)] = (uint8_t)sb;
}

// One unit out: e2m1 times E4M3 has six significant bits and lies within 2^-10 .. 2688,
// so all three types hold it exactly.
template <int TYPE>
__device__ __forceinline__ void store8(void* out, long long at, uint32_t codes, float s) {
    typedef float f32x2v __attribute__((ext_vector_type(2)));
    typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));
    const f32x2v x[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0) * s,
                         __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1) * s,
                         __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2) * s,
                         __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3) * s};
    if constexpr (TYPE == XP_F32) {
        *(float4*)((float*)out + at) = float4{x[0].x, x[0].y, x[1].x, x[1].y};
        *(float4*)((float*)out + at + 4) = float4{x[2].x, x[2].y, x[3].x, x[3].y};
    } else {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = TYPE == XP_BF16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(x[j], b16x2))
                                   : __builtin_bit_cast(uint32_t, __builtin_convertvector(x[j], h16x2));
        *(uint4*)((uint16_t*)out + at) = uint4{o[0], o[1], o[2], o[3]};
    }
}

// Few rows: a workgroup takes 256 units of one row.
template <int TYPE>
__global__ __launch_bounds__(256) void append_row_kernel(Geo g, RowMap m, const void* __restrict__ k, long long ks,
                                                         const void* __restrict__ v, long long vs, uint8_t* __restrict__ cache) {
    const int row = blockIdx.x, n = blockIdx.y * 256 + threadIdx.x, per = g.kv_heads * g.groups * 4;
    if (n >= 2 * per) return;                        // per is a multiple of 8: quads stay whole
    const bool is_v = n >= per;
    const int w = is_v ? n - per : n, head = w / (g.groups * 4);
    float x[8];
    load8<TYPE>(is_v ? v : k, (long long)row * (is_v ? vs : ks) + 8 * w, x);
    int pos;
    const long long tile = place(g, m, row, sequence_of(m.cu, m.batch, row), pos);
    if (tile < 0) return;
    quantise(g, Unit{(w >> 2) % g.groups, w & 3, is_v}, x, cache + tile + head * head_step(g), pos);
}
template <int TYPE>
__global__ __launch_bounds__(256) void read_row_kernel(Geo g, RowMap m, const uint8_t* __restrict__ cache, void* __restrict__ k,
                                                       long long ks, void* __restrict__ v, long long vs) {
    const int row = blockIdx.x, n = blockIdx.y * 256 + threadIdx.x, per = g.kv_heads * g.groups * 4;
    if (n >= 2 * per) return;
    const bool is_v = n >= per;
    const int w = is_v ? n - per : n, head = w / (g.groups * 4);
    const Unit u{(w >> 2) % g.groups, w & 3, is_v};
    int pos;
    const long long tile = place(g, m, row, sequence_of(m.cu, m.batch, row), pos);
    if (tile == -2) return;
    const uint8_t* t = cache + (tile < 0 ? 0 : tile + head * head_step(g));
    const uint32_t codes = tile < 0 ? 0u : *(const uint32_t*)(t + code_at(g, u, pos));
    const float s = tile < 0 ? 0.0f : e4m3_value(t[scale_at(g, u, pos)]);
    store8<TYPE>(is_v ? v : k, (long long)row * (is_v ? vs : ks) + 8 * w, codes, s);
}

// Many rows: a workgroup takes 64 rows of one kv head, so that the lines of a tile are
// written and read by one workgroup (or two, where rows and tiles are not aligned) and
// not by several chip parts with an L2 each. Bound by bytes: 2 (or 4) a value on one
// side, 4.25 bits on the other: 8,214 fp32 rows of 8 heads of 128 go in within 23 to
// 25 us (76 MB, 3.2 TB/s) and come out as bf16 in 12 us (43 MB, 3.5 TB/s); 32,768 rows
// come out in 30 us (170 MB, 5.6 TB/s). A workgroup for each row took 25, 18 and 60 us.
constexpr int kBlockRows = 64;
constexpr int kBatchRows = 4;   // rows a thread has in flight
struct Block {
    int units, rows_each;       // units of a kv head (of k and v), rows the workgroup takes at once
};
__device__ __forceinline__ Block block_of(const Geo& g) { return Block{8 * g.groups, 256 / (8 * g.groups)}; }
__device__ __forceinline__ void find_places(const Geo& g, const RowMap& m, int row0, long long* tile, int* pos) {
    if (threadIdx.x < kBlockRows) {
        int p;
        tile[threadIdx.x] = place(g, m, row0 + threadIdx.x, sequence_of(m.cu, m.batch, row0), p);
        pos[threadIdx.x] = p;
    }
    __syncthreads();
}

template <int TYPE>
__global__ __launch_bounds__(256) void append_block_kernel(Geo g, RowMap m, const void* __restrict__ k, long long ks,
                                                           const void* __restrict__ v, long long vs, uint8_t* __restrict__ cache) {
    __shared__ long long tile[kBlockRows];
    __shared__ int pos[kBlockRows];
    const int row0 = (int)(blockIdx.x / g.kv_heads) * kBlockRows, head = blockIdx.x % g.kv_heads;
    const Block bl = block_of(g);
    const int n = threadIdx.x % bl.units, r0 = threadIdx.x / bl.units;
    const Unit u{(n >> 2) % g.groups, n & 3, n >= 4 * g.groups};
    const void* src = u.is_v ? v : k;
    const long long stride = u.is_v ? vs : ks, col = (long long)head * g.groups * 32 + 8 * (n % (4 * g.groups));
    const long long hs = head * head_step(g);
    find_places(g, m, row0, tile, pos);
    for (int r = r0; r < kBlockRows; r += kBatchRows * bl.rows_each) {
        float x[kBatchRows][8];
#pragma unroll
        for (int i = 0; i < kBatchRows; ++i)         // 64 rows are whole batches for every head_dim
            if (tile[r + i * bl.rows_each] >= 0) load8<TYPE>(src, (row0 + r + i * bl.rows_each) * stride + col, x[i]);
#pragma unroll
        for (int i = 0; i < kBatchRows; ++i) {
            const long long t = tile[r + i * bl.rows_each];
            if (t >= 0) quantise(g, u, x[i], cache + t + hs, pos[r + i * bl.rows_each]);
        }
    }
}
template <int TYPE>
__global__ __launch_bounds__(256) void read_block_kernel(Geo g, RowMap m, const uint8_t* __restrict__ cache,
                                                         void* __restrict__ k, long long ks, void* __restrict__ v, long long vs) {
    __shared__ long long tile[kBlockRows];
    __shared__ int pos[kBlockRows];
    const int row0 = (int)(blockIdx.x / g.kv_heads) * kBlockRows, head = blockIdx.x % g.kv_heads;
    const Block bl = block_of(g);
    const int n = threadIdx.x % bl.units, r0 = threadIdx.x / bl.units;
    const Unit u{(n >> 2) % g.groups, n & 3, n >= 4 * g.groups};
    void* out = u.is_v ? v : k;
    const long long stride = u.is_v ? vs : ks, col = (long long)head * g.groups * 32 + 8 * (n % (4 * g.groups));
    const long long hs = head * head_step(g);
    find_places(g, m, row0, tile, pos);
    for (int r = r0; r < kBlockRows; r += kBatchRows * bl.rows_each) {
        uint32_t codes[kBatchRows];
        uint8_t sb[kBatchRows];
#pragma unroll
        for (int i = 0; i < kBatchRows; ++i) {
            const long long t = tile[r + i * bl.rows_each];
            const int p = pos[r + i * bl.rows_each];
            codes[i] = t < 0 ? 0u : *(const uint32_t*)(cache + t + hs + code_at(g, u, p));
            sb[i] = t < 0 ? (uint8_t)0 : cache[t + hs + scale_at(g, u, p)];
        }
#pragma unroll
        for (int i = 0; i < kBatchRows; ++i)
            if (tile[r + i * bl.rows_each] != -2)
                store8<TYPE>(out, (row0 + r + i * bl.rows_each) * stride + col, codes[i], e4m3_value(sb[i]));
    }
}

// Whether rows fill two workgroups of 64 on each of the 256 CUs.
static bool many_rows(const Geo& g, int rows) { return (long long)rows / kBlockRows * g.kv_heads >= 512; }

// ------------------------------------------------------------------ eviction
constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kSelKeys = 32768;     // positions whose keys are held in LDS; longer sequences read theirs again

// Weights in the order of selection as unsigned keys: larger first, -0 as +0,
// NaN below every number.
__device__ __forceinline__ uint32_t weight_key(float w) {
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
    if (u == 0x80000000u) u = 0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One workgroup per (sequence, kv head): the positions to keep, ascending. The key of
// the last one kept among the unprotected positions is found by three counting passes,
// of 12, 10 and 10 bits: the first takes sign, exponent and three bits of the
// significand, so weights that fall off over many powers of two spread over its bins.
// Then each wave walks its own run of positions, once to count and once to write.
// Bound by its own steps: 26 us for 64 of them over up to 16,384 positions (four passes
// of eight bits over keys in memory took 36 us), 10 us for eight over 1,100.
__global__ __launch_bounds__(kSelThreads) void evict_select_kernel(Geo g, const int32_t* __restrict__ lens,
                                                                   const float* weights, long long w_stride, int keep,
                                                                   int sinks, int recent, int32_t* kept,
                                                                   float* weights_out, long long wo_stride, int wo_len) {
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t bins[4096];
    __shared__ int part[kSelWaves];
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
        const bool any = want > 0, held_keys = n <= kSelKeys;
        uint32_t key = 0;                         // of the last one kept
        if (any) {
            if (held_keys)
                for (int i0 = lo; i0 < hi; i0 += 16 * kSelThreads) {
                    float x[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = i0 + j * kSelThreads + tid < hi ? w[i0 + j * kSelThreads + tid] : 0.0f;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (i0 + j * kSelThreads + tid < hi) keys[i0 + j * kSelThreads + tid] = weight_key(x[j]);
                }
            uint32_t known = 0;                   // its leading bits that are known
#pragma unroll 1
            for (int pass = 0; pass < 3; ++pass) {
                const int shift = pass == 0 ? 20 : (pass == 1 ? 10 : 0), each = pass == 0 ? 4 : 1;
                const uint32_t mask = pass == 0 ? 4095u : 1023u;
                for (int i = tid; i < 4096; i += kSelThreads) bins[i] = 0;
                __syncthreads();
                for (int i = lo + tid; i < hi; i += kSelThreads) {
                    const uint32_t k = held_keys ? keys[i] : weight_key(w[i]);
                    if ((k & known) == key) atomicAdd(&bins[(k >> shift) & mask], 1u);
                }
                __syncthreads();
                // a thread has `each` bins; `above`: counts of all the bins over its own
                int own = 0;
                for (int j = 0; j < each; ++j) own += (int)bins[tid * each + j];
                const int upto = wave_incl_sum(own);
                if (lane == 63) part[wave] = upto;
                __syncthreads();
                int above = part[wave] - upto;
                for (int j = wave + 1; j < kSelWaves; ++j) above += part[j];
                for (int j = each - 1; j >= 0; --j) {
                    const int t = (int)bins[tid * each + j];
                    if (above < want && above + t >= want) {
                        pick[0] = tid * each + j;
                        pick[1] = want - above;
                    }
                    above += t;
                }
                __syncthreads();
                key |= (uint32_t)pick[0] << shift;
                known |= mask << shift;
                want = pick[1];
            }
        }
        // want: how many of the positions that hold exactly `key` are kept, the lowest first
        const int run = ((n + kSelThreads - 1) / kSelThreads) * 64;
        const int from = wave * run, to = from + run < n ? from + run : n;
        int over = 0, tie = 0;
        for (int i0 = from; i0 < to; i0 += 64) {
            const int i = i0 + lane;
            const bool in = i < to, held = in && (i < lo || i >= hi), free = any && in && !held;
            const uint32_t k = free ? (held_keys ? keys[i] : weight_key(w[i])) : 0u;
            over += __popcll(__ballot(held || (free && k > key)));
            tie += __popcll(__ballot(free && k == key));
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
            const bool in = i < to, held = in && (i < lo || i >= hi), free = any && in && !held;
            const uint32_t k = free ? (held_keys ? keys[i] : weight_key(w[i])) : 0u;
            const bool is_tie = free && k == key;
            const uint64_t bt = __ballot(is_tie);
            const bool yes = held || (free && k > key) || (is_tie && ties + __popcll(bt & below) < want);
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

constexpr int kMoveThreads = 1024;
constexpr int kMoveSteps = 4;

// One workgroup per (group of 32 values of k or v, kv head, sequence): its kept
// positions' codes and scale bytes, in order. As above a step's loads are done
// before its stores, and later steps read only behind them, so the destination
// pages may be the source's own. Bound by bytes (17 in and out a position) and,
// for few positions, by the chain kept -> page table -> bytes of each step: a batch cut
// to a quarter takes 33 to 38 us, for the kept positions lie in most of the source's
// lines (103 MB fetched for 36 MB kept, and 36 MB written).
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
    if (rows < 0 || rows > 0x7fffffff - 64 || type < XP_BF16 || type > XP_F32) return XP_ERR_SHAPE;
    // a launch has fewer than 2^32 threads, 256 for 64 rows of a kv head
    if (((int64_t)rows + kBlockRows - 1) / kBlockRows * dims->kv_heads >= (1 << 24)) return XP_ERR_SHAPE;
    if (rows == 0 || batch == 0) return XP_OK;
    if (!k || !v || !cu || !start || !table || !cache) return XP_ERR_NULL;
    const int64_t width = (int64_t)dims->kv_heads * dims->head_dim, unit = type == XP_F32 ? 4 : 8;
    if (ks < width || vs < width || ks % unit || vs % unit) return XP_ERR_SHAPE;
    if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(cache, 16) || !aligned_to(cu, 4) || !aligned_to(start, 4) ||
        !aligned_to(table, 4))
        return XP_ERR_SHAPE;
    return XP_OK;
}

#define XP_ROWS_LAUNCH(KERNEL_, TYPE_, ...)                                                                              \
    do {                                                                                                                 \
        if (many_rows(g, rows))                                                                                          \
            hipLaunchKernelGGL(KERNEL_##_block_kernel<TYPE_>,                                                            \
                               dim3((unsigned)g.kv_heads * (unsigned)((rows + kBlockRows - 1) / kBlockRows)), dim3(256), \
                               0, s, __VA_ARGS__);                                                                       \
        else                                                                                                             \
            hipLaunchKernelGGL(KERNEL_##_row_kernel<TYPE_>,                                                              \
                               dim3((unsigned)rows, (unsigned)((8 * g.kv_heads * g.groups + 255) / 256)), dim3(256), 0, s, \
                               __VA_ARGS__);                                                                             \
    } while (0)

XP_API int xp_kv_append(const xp_kv_dims* dims, int32_t batch, int32_t max_pages, int32_t rows, int32_t type, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, const int32_t* cu_rows, const int32_t* start,
                        const int32_t* table, uint8_t* cache, void* stream) {
    const int st = check_rows(dims, batch, max_pages, rows, type, k, k_stride, v, v_stride, cu_rows, start, table, cache);
    if (st != XP_OK) return st;
    if (rows == 0 || batch == 0) return XP_OK;
    const Geo g = geo_of(dims, max_pages);
    const RowMap m{cu_rows, start, table, batch, rows};
    hipStream_t s = (hipStream_t)stream;
#define XP_APPEND(TYPE_)                                                                                                 \
    XP_ROWS_LAUNCH(append, TYPE_, g, m, k, (long long)k_stride, v, (long long)v_stride, cache)
    if (type == XP_BF16)
        XP_APPEND(XP_BF16);
    else if (type == XP_F16)
        XP_APPEND(XP_F16);
    else
        XP_APPEND(XP_F32);
#undef XP_APPEND
    return launch_status();
}

XP_API int xp_kv_read(const xp_kv_dims* dims, int32_t batch, int32_t max_pages, int32_t rows, int32_t type,
                      const int32_t* cu_rows, const int32_t* start, const int32_t* table, const uint8_t* cache, void* k,
                      int64_t k_stride, void* v, int64_t v_stride, void* stream) {
    const int st = check_rows(dims, batch, max_pages, rows, type, k, k_stride, v, v_stride, cu_rows, start, table, cache);
    if (st != XP_OK) return st;
    if (rows == 0 || batch == 0) return XP_OK;
    const int64_t size = type == XP_F32 ? 4 : 2, width = (int64_t)dims->kv_heads * dims->head_dim * size;
    if (rows_meet(Rows{k, rows, k_stride * size, width}, Rows{v, rows, v_stride * size, width})) return XP_ERR_SHAPE;
    const Geo g = geo_of(dims, max_pages);
    const RowMap m{cu_rows, start, table, batch, rows};
    hipStream_t s = (hipStream_t)stream;
#define XP_READ(TYPE_) XP_ROWS_LAUNCH(read, TYPE_, g, m, cache, k, (long long)k_stride, v, (long long)v_stride)
    if (type == XP_BF16)
        XP_READ(XP_BF16);
    else if (type == XP_F16)
        XP_READ(XP_F16);
    else
        XP_READ(XP_F32);
#undef XP_READ
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
    if (keep > (int64_t)0x80000000 - 8 * kSelThreads) return XP_ERR_SHAPE;   // indexes of the kernels' steps are ints
    if (batch == 0) return XP_OK;
    if (!cache || !table || !lens || !weights || !dst_table || !kept || !lens_out || !weights_out) return XP_ERR_NULL;
    if (w_stride < (int64_t)max_pages * dims->page || wo_stride < keep || !aligned_to(cache, 16) || !aligned_to(table, 4) ||
        !aligned_to(lens, 4) || !aligned_to(weights, 4) || !aligned_to(dst_table, 4) || !aligned_to(kept, 4) ||
        !aligned_to(lens_out, 4) || !aligned_to(weights_out, 4))
        return XP_ERR_SHAPE;
    // in place a row's weights are read before they are written; other overlaps would meet other rows' sources
    const int64_t most = (int64_t)max_pages * dims->page, n_rows = (int64_t)batch * dims->kv_heads;
    const Rows wr{weights, n_rows, 4 * w_stride, 4 * most}, wor{weights_out, n_rows, 4 * wo_stride, 4 * (most < wo_stride ? most : wo_stride)};
    if ((weights_out == weights && wo_stride != w_stride) || (!wr.same(wor) && rows_meet(wr, wor))) return XP_ERR_SHAPE;
    const Geo g = geo_of(dims, max_pages), d = geo_of(dims, dst_pages);
    hipStream_t s = (hipStream_t)stream;
    const int wo_len = wo_stride > 0x7fffffff ? 0x7fffffff : (int)wo_stride;
    const unsigned held = (unsigned)(most < kSelKeys ? most : kSelKeys) * sizeof(uint32_t);
    hipLaunchKernelGGL(evict_select_kernel, dim3(g.kv_heads, batch), dim3(kSelThreads), held, s, g, lens, weights,
                       (long long)w_stride, keep, sinks, recent, kept, weights_out, (long long)wo_stride, wo_len);
    const int rc = launch_status();
    if (rc != XP_OK) return rc;
    hipLaunchKernelGGL(evict_move_kernel, dim3(2 * g.groups, g.kv_heads, batch), dim3(kMoveThreads), 0, s, g, d, lens, table,
                       dst_table, kept, keep, cache, lens_out);
    return launch_status();
}
