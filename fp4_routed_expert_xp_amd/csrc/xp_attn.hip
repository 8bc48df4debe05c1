// xp_attn.hip — attention of a few query rows per sequence over the 4-bit cache.
//
// For each sequence and kv head, row r (query token r / group, head r % group of
// the kv head's group) holds softmax(scale * q . k) over the positions it sees,
// times v, in one pass over the cache with a running maximum and sum.
//
// One wave takes 64 positions at a time. Scores are formed transposed,
// S^T = K Q^T (v_mfma_f32_16x16x32_f16, K's positions as the rows), which leaves
// lane (c, q) = (lane % 16, lane / 16) with query row c at positions
// 16 t + 4 q + i (t, i = 0..3): the exponentials, once rounded to fp16, are then
// already the operand of O^T += V^T P^T with no movement between lanes, since the
// order of positions inside a contraction is free as long as V follows it. V's
// codes pass through LDS for that: a 4-bit transposing read hands each lane 16
// positions of one of V's columns in just that order.
//
// Precision: codes times scales are exact in fp16 (six significant bits). q in
// bf16 is scaled by a power of two to fp16, row by row, which is exact for every
// value within 2^28 of its row's largest. Scores, maxima, sums and outputs are
// fp32. The maximum is kept as the score it is, and the factor to log2 units multiplies
// differences only: the largest exponential is then 2^15 exactly for scores of any size
// (a maximum in log2 units has steps of 2 from 2^24 on, which fp16 does not survive).
// Exponentials round once to fp16 (2^-11), held as 2^15 p: what falls below
// fp16's normal numbers is then within 2^-40 of the row's largest.
//
// Bound by the cache's bytes where contexts are long: 64 ragged sequences to 8,192
// positions (8 kv heads of 128, 313 MB) take 79 us, 4.0 TB/s, 1.005 times the bytes
// fetched; 64 equal ones of 18,432 positions run at 5.7 TB/s. What is lost is mostly the
// longest sequence's chain of tiles, about 2.3 us each for its wave. The next tile's page
// number is part of that chain: it is loaded at the top of a tile and waited for, and with
// it the tile's V, which is needed only behind the scores. Per tile and wave
// the vector pipe issues some 440 instructions (256 of them decode codes and scales)
// and the matrix pipe 32 products: about half of the memory's time. Short calls are
// bound by the chain length -> page -> bytes -> products -> join, 8 us in all.
#include "xp_attn_dev.h"

namespace xp {
namespace attn {

using kv::Geo;

struct Args {
    Geo g;
    const void* q;
    long long q_stride;
    const uint8_t* cache;
    const int32_t* table;
    const int32_t* lens;
    void* out;
    long long out_stride;
    float* part;          // partial outputs of cut sequences' pieces, unscaled
    float* part_ml;       // their maxima (of the scores as they are formed), sums and the rows' factors
    float2* stats;        // per row, for the weights: the maximum of its scores and 1 / sum
    float* weights;
    long long w_stride;
    int heads, group, q_rows, row_blocks, window;
    int batch;
    int share, chunk;     // sequences longer than max(tiles of the batch / share, chunk) tiles are cut into pieces
    int waves;            // of a workgroup; pieces are whole rounds of them
    bool in_order;        // no sequence is cut, and units follow the grid
    float scale_m;        // scale * log2(e) = scale_m * 2^scale_e
    int scale_e;
};

// Query rows of a block of 16*MT: as they are,
template <int D, int MT>
__device__ __forceinline__ void fetch_q(const Args& a, int b, int head, int rb, int c, int q, uint4 (&v)[MT][Dim<D>::NW]) {
    const int rows = a.q_rows * a.group;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = (rb * MT + mt) * 16 + c;
        const bool ok = r < rows;
        const int tok = ok ? r / a.group : 0;
        const int hd = head * a.group + (ok ? r - tok * a.group : 0);
        const uint16_t* p = (const uint16_t*)a.q + ((long long)b * a.q_rows + tok) * a.q_stride + (long long)hd * D;
#pragma unroll
        for (int w = 0; w < Dim<D>::NW; ++w) v[mt][w] = ok ? *(const uint4*)(p + dims_of<D>(q, w)) : uint4{0, 0, 0, 0};
    }
}
// and as fp16 fragments, with each row's score factor.
template <int D, int MT, bool BF16>
__device__ __forceinline__ void make_q(const Args& a, const uint4 (&v)[MT][Dim<D>::NW], h16x8 (&qf)[MT][Dim<D>::NW],
                                       float (&factor)[MT]) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        int k = 0;
        if constexpr (BF16) {
            uint32_t top = 0;                   // exponent field of the row's largest magnitude
#pragma unroll
            for (int w = 0; w < Dim<D>::NW; ++w) {
                const uint32_t u[4] = {v[mt][w].x, v[mt][w].y, v[mt][w].z, v[mt][w].w};
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
                const uint32_t u[4] = {v[mt][w].x, v[mt][w].y, v[mt][w].z, v[mt][w].w};
                h16x8 f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = (_Float16)(__uint_as_float(u[i] << 16) * up);
                    f[2 * i + 1] = (_Float16)(__uint_as_float(u[i] & 0xffff0000u) * up);
                }
                qf[mt][w] = f;
            }
        } else {
#pragma unroll
            for (int w = 0; w < Dim<D>::NW; ++w) qf[mt][w] = __builtin_bit_cast(h16x8, v[mt][w]);
        }
        // kept a normal number: a masked -inf times 0, or a score of 0 times infinity, would be NaN
        factor[mt] = fminf(fmaxf(__builtin_amdgcn_ldexpf(a.scale_m, a.scale_e - k), 0x1p-126f), 0x1p127f);
    }
}

// Positions a row sees: from lo (inclusive) to hi (exclusive).
struct Span {
    int lo, hi;
};
__device__ __forceinline__ Span span_of(const Args& a, int len, int r) {
    const int rows = a.q_rows * a.group;
    const int at = len - a.q_rows + r / a.group;          // the row's own position
    Span s;
    s.hi = r < rows ? at + 1 : 0;
    s.lo = kv::first_seen(at, a.window);
    return s;
}

struct Tiles {
    int lo, hi;
};
__device__ __forceinline__ Tiles tiles_of(const Args& a, int len, int first_row, int last_row) {
    const Span first = span_of(a, len, first_row), last = span_of(a, len, last_row);
    Tiles t;
    t.lo = first.lo >> 6;
    t.hi = last.hi > 0 ? (last.hi + 63) >> 6 : 0;
    if (t.hi < t.lo) t.hi = t.lo;
    return t;
}

__device__ __forceinline__ int length_of(const Args& a, int b) {
    const int cap = a.g.max_pages * a.g.page;
    const int n = a.lens[b];
    return n < 0 ? 0 : (n > cap ? cap : n);
}

// The pieces of a launch. A unit is a (sequence, kv head, row block); a sequence's
// units are cut alike, into pieces that no more than one of `share` workgroups' even
// share of all tiles makes long, and sequences that are short enough are left whole.
// Cut sequences come first, then the whole ones, in batches of up to 64 the longer
// ones first, so that the short ones fill the gaps at the end. There are at
// most 2 * share pieces of cut sequences and share + units pieces in all.
struct Piece {
    int b, unit;          // sequence; kv head + kv_heads * row block
    int pieces, slot;     // pieces of the sequence; place of this unit's first one, kv_heads * row_blocks apart
    int tiles, lo, each;  // tiles of the sequence, the first one, tiles of a piece
    int index;            // which piece
    int len;
};
struct Cut {
    int tiles, lo, pieces, each;
};
__device__ __forceinline__ Cut cut_of(const Args& a, int len, int limit) {
    const Tiles t = tiles_of(a, len, 0, a.q_rows * a.group - 1);
    Cut c;
    c.lo = t.lo;
    c.tiles = t.hi - t.lo;
    c.pieces = c.tiles > limit ? (c.tiles + limit - 1) / limit : 1;
    c.each = (c.tiles + c.pieces - 1) / c.pieces;
    return c;
}
__device__ __forceinline__ int limit_of(const Args& a, long long even) {
    const int n = even > a.chunk ? (even > (1 << 26) ? 1 << 26 : (int)even) : a.chunk;
    return (n + a.waves - 1) / a.waves * a.waves;
}
// Piece i of the launch (JOIN: unit i of the cut sequences); false: there is none.
template <bool JOIN>
__device__ __forceinline__ bool find_piece(const Args& a, int i, Piece& p) {
    const int lane = threadIdx.x & 63, per = a.g.kv_heads * a.row_blocks;
    int limit = 0x7fffffff, len = 0;
    // a sequence's last piece is half empty on average: keep the pieces within one for each workgroup
    const long long units = (long long)a.batch * per, share = a.share - (units < a.share ? units : a.share) / 2;
    Cut c{};
    if (a.batch <= 64) {
        const bool in = lane < a.batch;
        len = in ? length_of(a, lane) : 0;
        c = cut_of(a, len, limit);
        if (a.share) {
            const int sum = wave_incl_sum(in ? c.tiles : 0);
            const long long all = (long long)(uint32_t)__builtin_amdgcn_readlane(sum, 63) * per;   // 64 * 2^25 tiles at most
            const long long even = (all + share - 1) / share;
            limit = limit_of(a, even);
            if (__ballot(in && c.tiles > limit)) c = cut_of(a, len, limit);
        }
        const bool is_cut = in && c.pieces > 1;
        const uint64_t cuts = __ballot(is_cut);
        int from = 0, first = 0;                           // pieces before this sequence's; (JOIN) units
        if (cuts) {
            first = wave_incl_sum(is_cut ? c.pieces * per : 0);
            from = __builtin_amdgcn_readlane(first, 63);
            first -= is_cut ? c.pieces * per : 0;
        }
        uint64_t hit;
        if (JOIN) {
            const int j = __popcll(cuts & ((1ull << lane) - 1)) * per;
            hit = __ballot(is_cut && j <= i && i < j + per);
            i -= j;                                        // per lane: read back from the one that hit
        } else {
            if (i >= from + (a.batch - __popcll(cuts)) * per) return false;
            if (i < from) {
                hit = __ballot(is_cut && first <= i && i < first + c.pieces * per);
                i -= first;
            } else {
                // eight classes of length, the longest first (top + 1 is top from 2^24 on)
                const int top = (int)wave_max_u32(in && !is_cut ? (uint32_t)c.tiles : 0u);
                const int part = top > 0 ? (int)(8.0f * (float)c.tiles / (float)(top + 1)) : 0;
                const int cls = in && !is_cut ? (part > 7 ? 7 : part) : -1;
                int before = 0;
#pragma unroll
                for (int k = 7; k >= 0; --k) {
                    const uint64_t same = __ballot(cls == k);
                    if (cls > k) continue;
                    before += __popcll(cls == k ? same & ((1ull << lane) - 1) : same);
                }
                first = from + before * per;
                hit = __ballot(cls >= 0 && first <= i && i < first + per);
                i -= first;
            }
        }
        if (!hit) return false;
        const int l = __ffsll((unsigned long long)hit) - 1;
        p.b = l;
        const int at = __builtin_amdgcn_readlane(i, l);
        p.index = JOIN ? 0 : at / per;
        p.unit = at - p.index * per;
        p.pieces = __builtin_amdgcn_readlane(c.pieces, l);
        p.slot = __builtin_amdgcn_readlane(first, l) + p.unit;
        p.tiles = __builtin_amdgcn_readlane(c.tiles, l);
        p.lo = __builtin_amdgcn_readlane(c.lo, l);
        p.each = __builtin_amdgcn_readlane(c.each, l);
        p.len = __builtin_amdgcn_readlane(len, l);
        return true;
    }
    // more sequences: their order is kept inside the cut and the whole ones
    {
        long long all = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 64) {
            c = cut_of(a, b0 + lane < a.batch ? length_of(a, b0 + lane) : 0, limit);
            const int v = wave_incl_sum(b0 + lane < a.batch ? c.tiles : 0);
            all += (uint32_t)__builtin_amdgcn_readlane(v, 63);
        }
        const long long even = (all * per + share - 1) / share;
        limit = limit_of(a, even);
    }
    int start = 0, jstart = 0;
    for (int whole = 0; whole < (JOIN ? 1 : 2); ++whole)
        for (int b0 = 0; b0 < a.batch; b0 += 64) {
            const bool in = b0 + lane < a.batch;
            len = in ? length_of(a, b0 + lane) : 0;
            c = cut_of(a, len, limit);
            const bool sel = in && (c.pieces == 1) == (whole == 1);
            const int mine = sel ? c.pieces * per : 0, joins = sel ? per : 0;
            const int incl = wave_incl_sum(mine), jincl = wave_incl_sum(joins);
            const int from = JOIN ? jstart + jincl - joins : start + incl - mine, n = JOIN ? joins : mine;
            const uint64_t hit = __ballot(sel && from <= i && i < from + n);
            if (hit) {
                const int l = __ffsll((unsigned long long)hit) - 1;
                p.b = b0 + l;
                const int at = i - __builtin_amdgcn_readlane(from, l);
                p.index = JOIN ? 0 : at / per;
                p.unit = at - p.index * per;
                p.pieces = __builtin_amdgcn_readlane(c.pieces, l);
                p.slot = start + __builtin_amdgcn_readlane(incl - mine, l) + p.unit;
                p.tiles = __builtin_amdgcn_readlane(c.tiles, l);
                p.lo = __builtin_amdgcn_readlane(c.lo, l);
                p.each = __builtin_amdgcn_readlane(c.each, l);
                p.len = __builtin_amdgcn_readlane(len, l);
                return true;
            }
            start += __builtin_amdgcn_readlane(incl, 63);
            jstart += __builtin_amdgcn_readlane(jincl, 63);
        }
    return false;
}

// A row's statistics for the weights kernel, which forms 2^((s - maximum) factor) times the
// second: kept apart, for one number in log2 units would round the sum's logarithm to the last
// place of the maximum. A row that sees nothing weighs nothing (its scores less infinity).
__device__ __forceinline__ float2 stats_of(float m, float l) {
    return l == 0.0f ? float2{__builtin_inff(), 0.0f} : float2{m, __builtin_amdgcn_ldexpf(1.0f / l, (int)kLift)};
}

// Waves a CU holds at once, by registers: also the most a workgroup takes. At 64 columns 131,072
// positions of 4 kv heads take 21.7 us in 16 and 20.0 in 12, 16 sequences to 2,500 positions 12.8
// and 14.1. Two sixteens of rows at 128 columns take 238 registers in 8 (16 sequences to 8,192
// positions, 8 kv heads, 40 rows: 59 us) and, left to grow, 324 in 4 (85 us).
template <int D, int MT>
constexpr int waves_per_cu() {
    return MT == 1 ? (D == 64 ? 16 : (D == 128 ? 12 : 8)) : 8;
}
template <int D, int MT>
constexpr int region_bytes() {
    return Dim<D>::kVBytes + Dim<D>::NG * 64;              // a wave's V codes and scales
}
template <int D, int MT>
constexpr int join_bytes() {
    return MT * Dim<D>::NH * 1024 + MT * 128;              // a wave's output, maxima and sums
}

// One workgroup: a split of one (sequence, kv head, block of 16*MT rows); its waves
// take tiles in turn and join in LDS.
template <int D, int MT, bool BF16>
__global__ __launch_bounds__((64 * waves_per_cu<D, MT>())) void attn_decode_kernel(Args a) {
    constexpr int NW = Dim<D>::NW, NG = Dim<D>::NG, NH = Dim<D>::NH, VD = Dim<D>::VD;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    // In order, units follow the grid: q and the first page are asked for before the length is known.
    Piece pc;
    const int units = a.g.kv_heads * a.row_blocks, page_tiles = a.g.page >> 6;
    int first_id = -1;
    uint4 qv[MT][NW];
    if (a.in_order) {
        pc.b = blockIdx.x / units;
        pc.unit = blockIdx.x - pc.b * units;
        const int col = wave / page_tiles;
        first_id = a.table[(long long)pc.b * a.g.max_pages + (col < a.g.max_pages ? col : 0)];
        const int rb = pc.unit / a.g.kv_heads;
        fetch_q<D, MT>(a, pc.b, pc.unit - rb * a.g.kv_heads, rb, c, q, qv);
        pc.len = length_of(a, pc.b);
        const Cut cut = cut_of(a, pc.len, 0x7fffffff);
        pc.pieces = 1;
        pc.slot = pc.index = 0;
        pc.tiles = pc.each = cut.tiles;
        pc.lo = cut.lo;
    } else if (!find_piece<false>(a, blockIdx.x, pc)) {
        return;
    }
    const int b = pc.b, len = pc.len, rb = pc.unit / a.g.kv_heads, head = pc.unit - rb * a.g.kv_heads;
    const int32_t* tr = a.table + (long long)b * a.g.max_pages;
    if (!a.in_order) fetch_q<D, MT>(a, b, head, rb, c, q, qv);

    // this piece's tiles, less those that no row of the block sees
    const int rows = a.q_rows * a.group, first_row = rb * MT * 16;
    const int last_row = first_row + MT * 16 < rows ? first_row + MT * 16 - 1 : rows - 1;
    const Tiles tl = tiles_of(a, len, first_row, last_row);
    int t0 = pc.lo + pc.index * pc.each, t1 = t0 + pc.each;
    t1 = t1 > pc.lo + pc.tiles ? pc.lo + pc.tiles : t1;
    t0 = t0 < tl.lo ? tl.lo : t0;
    t1 = t1 > tl.hi ? tl.hi : t1;
    // positions that every row sees
    const int full_lo = span_of(a, len, last_row).lo, full_hi = span_of(a, len, first_row).hi;

    // a tile's bytes, asked for one tile ahead: K once its scores are formed, V once it is in LDS
    // (both have to be there when the page after them is known, see above)
    KTile<D> k;
    uint32_t vw[VD];
    constexpr int SW = NG * 64 / 4;                        // dwords of V scales
    uint32_t vs[(SW + 63) / 64];
    auto load_v = [&](const uint8_t* t) {
#pragma unroll
        for (int j = 0; j < VD / 4; ++j) {
            const uint4 v = *(const uint4*)(t + NG * 1088 + j * 1024 + lane * 16);
            vw[4 * j] = v.x;
            vw[4 * j + 1] = v.y;
            vw[4 * j + 2] = v.z;
            vw[4 * j + 3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < (SW + 63) / 64; ++j)
            vs[j] = j * 64 + lane < SW ? *(const uint32_t*)(t + NG * 2112 + (j * 64 + lane) * 4) : 0u;
    };
    // the next tile at or behind `tile` whose page exists (positions of others are not seen);
    // its page's column and its place on the page follow it
    const long long tile_bytes = kv::tile_bytes(NG);
    bool asked = a.in_order && t0 == 0;
    int tile = t0 + wave, col = tile / page_tiles, in_page = tile - col * page_tiles;
    auto find = [&](int& tile) {
        for (; tile < t1; tile += waves) {
            const int id = asked ? first_id : tr[col];
            asked = false;
            const long long at = (((long long)id * a.g.kv_heads + head) * page_tiles + in_page) * tile_bytes;
            for (in_page += waves; in_page >= page_tiles; in_page -= page_tiles) ++col;
            if ((unsigned)id < (unsigned)a.g.n_pages) return a.cache + at;
        }
        return a.cache;
    };
    const uint8_t* t = find(tile);
    if (tile < t1) {
        load_k<D>(k, t, c, q);
        load_v(t);
    }
    h16x8 qf[MT][NW];
    float factor[MT];
    make_q<D, MT, BF16>(a, qv, qf, factor);

    f32x4 o[MT][NH];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = -__builtin_inff();
        l[mt] = 0.0f;
#pragma unroll
        for (int h = 0; h < NH; ++h) o[mt][h] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    uint8_t* region = lds + wave * region_bytes<D, MT>();

    while (tile < t1) {
        int next = tile + waves;
        const uint8_t* nt = find(next);
        f32x4 s[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int bl = 0; bl < 4; ++bl) s[mt][bl] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int bl = 0; bl < 4; ++bl)
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const h16x8 kf = k_frag<D>(k, bl, w);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) s[mt][bl] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[mt][w], s[mt][bl], 0, 0, 0);
            }

        if (next < t1) load_k<D>(k, nt, c, q);

        const bool masked = tile * 64 < full_lo || tile * 64 + 64 > full_hi;
        bool nan_v = false;
        if (masked) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const Span sp = span_of(a, len, (rb * MT + mt) * 16 + c);
#pragma unroll
                for (int bl = 0; bl < 4; ++bl)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int pos = tile * 64 + 16 * bl + 4 * q + i;
                        if (pos < sp.lo || pos >= sp.hi) s[mt][bl][i] = -__builtin_inff();
                    }
            }
            // V where not every row sees it: bytes behind the sequence are no values, and a
            // NaN scale must not reach rows that do not see its position
#pragma unroll
            for (int j = 0; j < (SW + 63) / 64; ++j) {
                const int at_byte = (j * 64 + lane) * 4;   // byte 4x + y of a group: position 16 (x % 4) + 4 (x / 4) + y
                const int x = (at_byte & 63) >> 2;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int pos = tile * 64 + 16 * (x & 3) + 4 * (x >> 2) + y;
                    if (pos >= len) vs[j] &= ~(255u << (8 * y));
                    if (((vs[j] >> (8 * y)) & 127u) == 127u) nan_v = true;
                }
            }
            nan_v = __ballot(nan_v) != 0;
        }

        // V to LDS; this wave's earlier reads of the region are done (LDS keeps a wave's order)
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < VD / 4; ++j)
            *(uint4*)(region + j * 1024 + lane * 16) = uint4{vw[4 * j], vw[4 * j + 1], vw[4 * j + 2], vw[4 * j + 3]};
#pragma unroll
        for (int j = 0; j < (SW + 63) / 64; ++j)
            if (j * 64 + lane < SW) *(uint32_t*)(region + Dim<D>::kVBytes + (j * 64 + lane) * 4) = vs[j];
        __builtin_amdgcn_wave_barrier();
        if (next < t1) load_v(nt);

        h16x8 p[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float mx = s[mt][0][0];
#pragma unroll
            for (int e = 1; e < 16; ++e) mx = fmaxf(mx, s[mt][e >> 2][e & 3]);
            mx = max_over_q(mx);
            if (__ballot(mx > m[mt])) {
                const float nm = fmaxf(mx, m[mt]);
                const float safe = nm == -__builtin_inff() ? 0.0f : nm;
                const float alpha = __builtin_amdgcn_exp2f((m[mt] - safe) * factor[mt]);
                m[mt] = nm;
                l[mt] *= alpha;
#pragma unroll
                for (int h = 0; h < NH; ++h) o[mt][h] *= alpha;
            }
            const float top = m[mt] == -__builtin_inff() ? 0.0f : m[mt];
            float add = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[mt][e >> 2][e & 3] - top, factor[mt], kLift));
                add += x;
                p[mt][e >> 3][e & 7] = (_Float16)x;
            }
            l[mt] += add;
        }

        if (masked && nan_v) {
            // a zero weight times a NaN scale is NaN: rows that see such a position get NaN in its
            // group's columns here, and the scale leaves the tile
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint8_t* sb = region + Dim<D>::kVBytes + g * 64 + q * 16;
                uint32_t bad = 0;
#pragma unroll 1
                for (int e = 0; e < 16; ++e) bad |= ((sb[e] & 127u) == 127u ? 1u : 0u) << e;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const Span sp = span_of(a, len, (rb * MT + mt) * 16 + c);
                    float hit = 0.0f;
#pragma unroll 1
                    for (int e = 0; e < 16; ++e) {
                        const int ps = tile * 64 + 16 * (e >> 2) + 4 * q + (e & 3);
                        if ((bad >> e & 1u) && ps >= sp.lo && ps < sp.hi) hit = 1.0f;
                    }
                    const float add = max_over_q(hit) > 0.0f ? __builtin_nanf("") : 0.0f;
                    o[mt][2 * g] += add;
                    o[mt][2 * g + 1] += add;
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll 1
                for (int e = 0; e < 16; ++e)
                    if (bad >> e & 1u) sb[e] = 0;
            }
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
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
                const int h = 2 * g + hh;
                const int pos = 16 * (c >> 2) + 4 * q + (c & 3);
                const i32x2 vt = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                    (__attribute__((address_space(3))) i32x2*)(region + h * 512 + pos * 8));
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    const h16x8 vf = decode8((uint32_t)vt[st], sv[4 * st], sv[4 * st + 1], sv[4 * st + 2], sv[4 * st + 3]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        o[mt][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[mt][st], o[mt][h], 0, 0, 0);
                }
            }
        }
        tile = next;
    }

    // join the waves: each leaves its share in LDS, then takes every waves-th column block
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) l[mt] = sum_over_q(l[mt]);
    __syncthreads();                                       // the regions are read
    int quarter = q;                                       // q, formed again: held over the loop, what is
    asm volatile("" : "+v"(quarter));                      // derived from it spills 64 columns' 128 registers
    {
        f32x4* buf = (f32x4*)(lds + wave * join_bytes<D, MT>());
        float* ml = (float*)(buf + MT * NH * 64);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int h = 0; h < NH; ++h) buf[(mt * NH + h) * 64 + lane] = o[mt][h];
            if (q == 0) {
                ml[mt * 32 + c] = m[mt];
                ml[mt * 32 + 16 + c] = l[mt];
            }
        }
    }
    __syncthreads();
    const long long slot = pc.slot + (long long)pc.index * (a.g.kv_heads * a.row_blocks);
    for (int col_block = wave; col_block < MT * NH; col_block += waves) {
        const int mt = MT == 1 ? 0 : col_block / NH, h = col_block - mt * NH;
        const float fr = mt == 0 ? factor[0] : factor[MT - 1];
        float jm = -__builtin_inff(), jl = 0.0f;
        for (int w = 0; w < waves; ++w)
            jm = fmaxf(jm, ((const float*)(lds + w * join_bytes<D, MT>() + MT * NH * 1024))[mt * 32 + c]);
        const float safe = jm == -__builtin_inff() ? 0.0f : jm;
        f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < waves; ++w) {
            const uint8_t* from = lds + w * join_bytes<D, MT>();
            const float* ml = (const float*)(from + MT * NH * 1024) + mt * 32 + c;
            const float f = __builtin_amdgcn_exp2f((ml[0] - safe) * fr);
            jl = __builtin_fmaf(ml[16], f, jl);
            acc += ((const f32x4*)from)[col_block * 64 + lane] * f;
        }
        if (pc.pieces > 1) {
            ((f32x4*)a.part)[(slot * (MT * NH) + col_block) * 64 + lane] = acc;
            float* pm = a.part_ml + slot * (MT * 48) + mt * 48 + c;
            if (h == 0 && q == 0) {
                pm[0] = jm;
                pm[16] = jl;
                pm[32] = fr;
            }
            continue;
        }
        const int r = (rb * MT + mt) * 16 + c;
        if (r >= rows) continue;
        const int tok = r / a.group, hd = head * a.group + r - tok * a.group;
        uint16_t* y = (uint16_t*)a.out + ((long long)b * a.q_rows + tok) * a.out_stride + (long long)hd * D;
        const float inv = jl == 0.0f ? 0.0f : 1.0f / jl;   // nothing seen: zeros
        *(uint2*)(y + 16 * h + 4 * quarter) = to16<BF16>(acc * inv);
        if (a.stats && h == 0 && q == 0) a.stats[((long long)b * a.heads + head * a.group) * a.q_rows + r] = stats_of(jm, jl);
    }
}

// Joins the pieces of a cut sequence: a workgroup takes four columns of 16 rows a lane,
// its waves take the pieces in turn (their partial outputs are 1 KiB loads that do not
// wait for each other) and meet in LDS, in order. 5 to 6 us; one wave over 256 pieces
// took 130 us.
constexpr int kJoinWaves = 16;
template <int D, int MT, bool BF16>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join_kernel(Args a) {
    constexpr int NH = Dim<D>::NH;
    __shared__ f32x4 so[kJoinWaves][64];
    __shared__ float sm[kJoinWaves][64], sl[kJoinWaves][64];
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int h = blockIdx.x % NH, mt = blockIdx.x / NH;
    Piece pc;
    if (!find_piece<true>(a, blockIdx.y, pc)) return;
    const int b = pc.b, rb = pc.unit / a.g.kv_heads, head = pc.unit - rb * a.g.kv_heads, n = pc.pieces;
    const long long step = a.g.kv_heads * a.row_blocks;    // slots from one piece of a unit to its next
    const f32x4* po = (const f32x4*)a.part + (long long)pc.slot * (MT * NH * 64) + blockIdx.x * 64 + lane;
    const float* pm = a.part_ml + (long long)pc.slot * (MT * 48) + mt * 48 + c;
    const float fr = pm[32];                               // the row's factor, the same with every piece
    float m = -__builtin_inff(), l = 0.0f;
    f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int U = 8;
    for (int s0 = wave; s0 < n; s0 += U * waves) {
        f32x4 v[U];
        float vm[U], vl[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * waves < n ? s0 + u * waves : s0;
            v[u] = po[s * step * (MT * NH * 64)];
            vm[u] = pm[s * step * (MT * 48)];
            vl[u] = pm[s * step * (MT * 48) + 16];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u * waves >= n) break;
            const float nm = fmaxf(m, vm[u]), safe = nm == -__builtin_inff() ? 0.0f : nm;
            const float fa = __builtin_amdgcn_exp2f((m - safe) * fr), fb = __builtin_amdgcn_exp2f((vm[u] - safe) * fr);
            m = nm;
            l = l * fa + vl[u] * fb;
            o = o * fa + v[u] * fb;
        }
    }
    so[wave][lane] = o;
    sm[wave][lane] = m;
    sl[wave][lane] = l;
    __syncthreads();
    const int r = (rb * MT + mt) * 16 + c;
    if (wave > 0 || r >= a.q_rows * a.group) return;
    for (int w = 1; w < waves; ++w) {
        const float om = sm[w][lane], nm = fmaxf(m, om), safe = nm == -__builtin_inff() ? 0.0f : nm;
        const float fa = __builtin_amdgcn_exp2f((m - safe) * fr), fb = __builtin_amdgcn_exp2f((om - safe) * fr);
        m = nm;
        l = l * fa + sl[w][lane] * fb;
        o = o * fa + so[w][lane] * fb;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int tok = r / a.group, hd = head * a.group + r - tok * a.group;
    uint16_t* y = (uint16_t*)a.out + ((long long)b * a.q_rows + tok) * a.out_stride + (long long)hd * D;
    *(uint2*)(y + 16 * h + 4 * q) = to16<BF16>(o * inv);
    if (a.stats && h == 0 && q == 0) a.stats[((long long)b * a.heads + head * a.group) * a.q_rows + r] = stats_of(m, l);
}

// weights[pos] += the probabilities of all rows of the kv head at pos, from each
// row's maximum and sum. Scores are formed with the rows first (S = Q K^T), so
// a lane adds four rows of one position by itself and two swaps add the rest; one
// wave owns a tile, so no atomics. K is read a second time: half the cache's bytes,
// against writing and reading every row's scores (as much for eight rows a head). 19 us
// for 8 ragged sequences to 16,384 positions of 8 kv heads (45 MB with the weights in
// and out, 2.4 TB/s), where a form that made q's fragments for every tile took 25 us.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void attn_weights_kernel(Args a) {
    constexpr int NW = Dim<D>::NW;
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.y, b = blockIdx.z;
    const int len = length_of(a, b);
    const int32_t* tr = a.table + (long long)b * a.g.max_pages;
    const int rows = a.q_rows * a.group;
    const int t_lo = span_of(a, len, 0).lo >> 6, t_hi = (len + 63) >> 6;
    const float2* stats = a.stats + ((long long)b * a.heads + head * a.group) * a.q_rows;
    float* weights = a.weights + ((long long)b * a.g.kv_heads + head) * a.w_stride;
    const int first = t_lo + blockIdx.x * 4 + wave, step = gridDim.x * 4;
    for (int rb = 0; rb * 16 < rows && first < t_hi; ++rb) {
        h16x8 qf[1][NW];
        float factor[1], f[4];
        float2 st[4];
        Span sp[4];
        KTile<D> k;
        long long at = kv::tile_at(a.g, tr, head, first * 64);
        load_k<D>(k, a.cache + (at < 0 ? 0 : at), c, q);
        uint4 qv[1][NW];
        fetch_q<D, 1>(a, b, head, rb, c, q, qv);
        make_q<D, 1, BF16>(a, qv, qf, factor);
        int all_lo = 0, all_hi = 0x7fffffff;               // positions that the lane's rows all see
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rb * 16 + 4 * q + i;
            f[i] = __shfl(factor[0], 4 * q + i);           // held by the lane whose c is the row
            st[i] = r < rows ? stats[r] : float2{__builtin_inff(), 0.0f};
            sp[i] = span_of(a, len, r);
            if (r >= rows) continue;                       // rows that are not there weigh nothing
            all_lo = sp[i].lo > all_lo ? sp[i].lo : all_lo;
            all_hi = sp[i].hi < all_hi ? sp[i].hi : all_hi;
        }
        for (int tile = first; tile < t_hi; tile += step) {
            const int next = tile + step;
            const long long next_at = next < t_hi ? kv::tile_at(a.g, tr, head, next * 64) : -1;
            f32x4 s[4];
#pragma unroll
            for (int bl = 0; bl < 4; ++bl) {
                s[bl] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int wd = 0; wd < NW; ++wd)
                    s[bl] = __builtin_amdgcn_mfma_f32_16x16x32_f16(qf[0][wd], k_frag<D>(k, bl, wd), s[bl], 0, 0, 0);
            }
            const bool there = at >= 0;
            at = next_at;
            if (next < t_hi) load_k<D>(k, a.cache + (at < 0 ? 0 : at), c, q);
            if (!there) continue;
            const int mine_at = tile * 64 + 16 * q + c;
            const float old = mine_at < len ? weights[mine_at] : 0.0f;
            float w[4] = {0.f, 0.f, 0.f, 0.f};
            const bool whole = __ballot(tile * 64 < all_lo || tile * 64 + 64 > all_hi) == 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int bl = 0; bl < 4; ++bl) {
                    const int pos = tile * 64 + 16 * bl + c;
                    const float e = __builtin_amdgcn_exp2f((s[bl][i] - st[i].x) * f[i]);
                    w[bl] = whole || (pos >= sp[i].lo && pos < sp[i].hi) ? __builtin_fmaf(e, st[i].y, w[bl]) : w[bl];
                }
            float mine = 0.0f;
#pragma unroll
            for (int bl = 0; bl < 4; ++bl) {
                const float t = sum_over_q(w[bl]);
                mine = q == bl ? t : mine;
            }
            if (mine_at < len) weights[mine_at] = old + mine;
        }
    }
}

// Rows of a block: 16 * MT. Two sixteens read a tile's bytes once and decode them once for both,
// with half as many registers again. 16 sequences to 8,192 positions of 8 kv heads, 128 columns, 32
// rows a kv head: 39 us (43 in blocks of 16); 40 rows: 59 (60); one of 65,536: 31 (33); at 64
// columns 27 (28). Where there are units enough without, blocks of 16 are faster: 32 sequences
// to 4,096 42 us (37), eight to 700 12.6 (10.5). At 256 columns two exceed the registers.
static int row_tiles(int rows, int dim) { return rows <= 16 || dim == 256 ? 1 : 2; }

constexpr int kCus = 256;
// With two units a CU or more, sequences of up to this many tiles are never cut.
constexpr int kLongTiles = 256;

struct Launch {
    int mt, row_blocks, waves, share, chunk, join_waves;
    long long units;
    size_t part, ml, stats, total;
};
// What a call with these arguments launches and keeps in its workspace (with a window
// no more than without: it only shortens what is seen).
static Launch plan_of(const xp_kv_dims* d, int heads, int q_rows, int batch, int max_len, int window) {
    Launch p{};
    const long long rows = (long long)q_rows * (heads / d->kv_heads);
    p.mt = row_tiles(rows > 64 ? 64 : (int)rows, d->head_dim);
    p.row_blocks = (int)((rows + 16 * p.mt - 1) / (16 * p.mt));
    long long blocks = (long long)batch * d->kv_heads * p.row_blocks;
    blocks = blocks < 1 ? 1 : blocks;
    long long tiles = max_len < 1 ? 1 : ((long long)max_len + 63) / 64;
    const long long seen = ((long long)window + q_rows + 62) / 64 + 1;
    tiles = window > 0 && seen < tiles ? seen : tiles;
    p.units = blocks;
    const int most = d->head_dim == 64 ? (p.mt == 1 ? waves_per_cu<64, 1>() : waves_per_cu<64, 2>())
                     : d->head_dim == 128 ? (p.mt == 1 ? waves_per_cu<128, 1>() : waves_per_cu<128, 2>())
                                          : waves_per_cu<256, 1>();
    // Contexts of a few rounds are left whole, by as many waves as there is room for. Longer
    // ones are cut into one workgroup of the most waves on each CU where there are few units
    // (one sequence of 131,072 positions, 4 kv heads: 25 us, against 29 in fours: fewer pieces
    // to join), else into workgroups of four waves, as many as it holds (16 ragged sequences to
    // 8,192, 8 kv heads: 29 us, against 31 in one of twelve; eight to 16,384 with weights 48.5
    // and 46.6, 48 to 8,192 67 and 64: within 6% either way).
    const bool many = blocks >= 2 * kCus, few = blocks <= 16, cut = tiles > (many ? kLongTiles : 3 * most);
    p.waves = many || (cut && !few) ? 4 : (int)(tiles < most ? tiles : most);
    p.chunk = many ? kLongTiles : 2 * p.waves;
    p.share = cut ? kCus * (few ? 1 : most / 4) : 0;          // 0: no sequence is cut
    const long long pieces = (tiles + p.chunk - 1) / p.chunk;
    p.join_waves = (int)(pieces > 4 * kJoinWaves ? kJoinWaves : (pieces + 3) / 4);
    const size_t parts = 2 * (size_t)p.share;
    p.part = 0;
    p.ml = parts * 16 * p.mt * d->head_dim * sizeof(float);
    p.stats = p.ml + align256(parts * 48 * p.mt * sizeof(float));
    p.total = p.stats + align256((size_t)batch * heads * q_rows * sizeof(float2));
    return p;
}

static int check_decode(const xp_kv_dims* d, int heads, int q_rows, int batch, int max_pages, int max_len) {
    const int st = kv::check_geo(d, batch, max_pages);
    if (st != XP_OK) return st;
    if (heads < 1 || heads > 65535 || heads % d->kv_heads || q_rows < 1 || q_rows > 65535 || max_len < 0) return XP_ERR_SHAPE;
    if ((long long)heads * q_rows > (1 << 24)) return XP_ERR_SHAPE;     // rows of a sequence fit an int
    const Launch p = plan_of(d, heads, q_rows, batch, max_len, 0);
    if (p.units > (1 << 22)) return XP_ERR_SHAPE;   // four waves each then: a launch has fewer than 2^32 threads
    return XP_OK;
}

template <int D, bool BF16>
static int launch(const Args& a, const Launch& p, int batch, int max_len, hipStream_t s) {
    const dim3 grid((unsigned)(p.units + p.share)), block(64 * p.waves);
    const dim3 join(p.mt * D / 16, (unsigned)(p.units < p.share ? p.units : p.share)), join_block(64 * p.join_waves);
#define XP_ATTN_LAUNCH(MT_)                                                                        \
    do {                                                                                           \
        const int per_wave = join_bytes<D, MT_>() > region_bytes<D, MT_>() ? join_bytes<D, MT_>() : region_bytes<D, MT_>(); \
        hipLaunchKernelGGL((attn_decode_kernel<D, MT_, BF16>), grid, block, p.waves * per_wave, s, a); \
        if (p.share) hipLaunchKernelGGL((attn_join_kernel<D, MT_, BF16>), join, join_block, 0, s, a); \
    } while (0)
    if (p.mt == 1)
        XP_ATTN_LAUNCH(1);
    else if constexpr (D != 256)
        XP_ATTN_LAUNCH(2);
#undef XP_ATTN_LAUNCH
    int rc = launch_status();
    if (rc != XP_OK || !a.weights) return rc;
    const long long tiles = ((long long)max_len + 63) / 64;
    // four waves a workgroup, three workgroups on each CU, at least a tile for each wave
    long long blocks = (3 * kCus + (long long)batch * a.g.kv_heads - 1) / ((long long)batch * a.g.kv_heads);
    blocks = blocks > (tiles + 3) / 4 ? (tiles + 3) / 4 : blocks;
    blocks = blocks < 1 ? 1 : blocks;
    hipLaunchKernelGGL((attn_weights_kernel<D, BF16>), dim3((unsigned)blocks, a.g.kv_heads, batch), dim3(256), 0, s, a);
    return launch_status();
}

}  // namespace attn
}  // namespace xp

using namespace xp;
using namespace xp::attn;

XP_API size_t xp_attn_decode_workspace_bytes(const xp_kv_dims* dims, int32_t heads, int32_t q_rows, int32_t batch,
                                             int32_t max_len) {
    if (check_decode(dims, heads, q_rows, batch, 1, max_len) != XP_OK) return 0;
    return plan_of(dims, heads, q_rows, batch, max_len, 0).total;
}

XP_API int xp_attn_decode(const xp_kv_dims* dims, int32_t heads, int32_t q_rows, int32_t batch, int32_t max_pages,
                          int32_t max_len, int32_t type, const void* q, int64_t q_stride, float scale, int32_t window,
                          const uint8_t* cache, const int32_t* table, const int32_t* lens, void* out, int64_t out_stride,
                          float* weights, int64_t w_stride, void* workspace, size_t ws_bytes, void* stream) {
    const int st = check_decode(dims, heads, q_rows, batch, max_pages, max_len);
    if (st != XP_OK) return st;
    if ((type != XP_BF16 && type != XP_F16) || window < 0 || !(scale > 0.0f && scale < __builtin_inff())) return XP_ERR_SHAPE;
    if (batch == 0) return XP_OK;
    if (!q || !cache || !table || !lens || !out || !workspace) return XP_ERR_NULL;
    const int64_t width = (int64_t)heads * dims->head_dim;
    if (q_stride < width || out_stride < width || q_stride % 8 || out_stride % 4 || !kv::aligned_to(q, 16) ||
        !kv::aligned_to(out, 8) || !kv::aligned_to(cache, 16) || !kv::aligned_to(table, 4) || !kv::aligned_to(lens, 4) ||
        !kv::aligned_to(workspace, 16))
        return XP_ERR_SHAPE;
    if (weights && (w_stride < (int64_t)max_pages * dims->page || !kv::aligned_to(weights, 4))) return XP_ERR_SHAPE;
    // a unit's q is read before its rows are written, but the weights kernel reads q again
    const kv::Rows qr{q, (int64_t)batch * q_rows, 2 * q_stride, 2 * width}, yr{out, qr.n, 2 * out_stride, 2 * width};
    if ((weights || !qr.same(yr)) && kv::rows_meet(qr, yr)) return XP_ERR_SHAPE;
    const Launch p = plan_of(dims, heads, q_rows, batch, max_len, window);
    if (ws_bytes < p.total) return XP_ERR_WORKSPACE;
    char* ws = (char*)workspace;
    Args a{};
    a.g = kv::geo_of(dims, max_pages);
    a.q = q;
    a.q_stride = q_stride;
    a.cache = cache;
    a.table = table;
    a.lens = lens;
    a.out = out;
    a.out_stride = out_stride;
    a.part = (float*)(ws + p.part);
    a.part_ml = (float*)(ws + p.ml);
    a.stats = weights ? (float2*)(ws + p.stats) : nullptr;
    a.weights = weights;
    a.w_stride = w_stride;
    a.heads = heads;
    a.group = heads / dims->kv_heads;
    a.q_rows = q_rows;
    a.row_blocks = p.row_blocks;
    a.batch = batch;
    a.share = p.share;
    a.waves = p.waves;
    // units that each have a CU, or of more sequences than a wave sorts, need no order
    a.in_order = !p.share && (p.units <= kCus || batch > 64);
    a.chunk = p.chunk;
    a.window = window;
    a.scale_m = (float)__builtin_frexp((double)scale * 1.4426950408889634, &a.scale_e);
    hipStream_t s = (hipStream_t)stream;
    const bool bf = type == XP_BF16;
    switch (dims->head_dim) {
        case 64: return bf ? launch<64, true>(a, p, batch, max_len, s) : launch<64, false>(a, p, batch, max_len, s);
        case 128: return bf ? launch<128, true>(a, p, batch, max_len, s) : launch<128, false>(a, p, batch, max_len, s);
        default: return bf ? launch<256, true>(a, p, batch, max_len, s) : launch<256, false>(a, p, batch, max_len, s);
    }
}
