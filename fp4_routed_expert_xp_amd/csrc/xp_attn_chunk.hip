// xp_attn_chunk.hip — attention of packed new tokens over the 4-bit cache: pieces of
// prompts behind any number of cached positions, single tokens among them.
//
// The products are those of prompt attention (xp_attn_prompt.hip): a row is a (token, head
// of the kv head's group) pair, a wave owns RW rows, scores are formed transposed, and the
// rounded exponentials are the second product's operand where they are. What differs is
// where keys and values come from: a tile's codes are loaded two tiles ahead into
// registers, a wave a kilobyte, and decoded one tile ahead into LDS, 16 bits a value, once
// for all rows of the workgroup.
//
// Precision: codes times scales are exact in fp16. q in bf16 is scaled by a power of two
// to fp16, row by row, exact within 2^28 of the row's largest. Scores, maxima, sums and
// outputs are fp32; exponentials round once to fp16 as 2^13 p, and sums are of the rounded
// ones; the maximum may lag by 2^2 (see xp_attn_prompt.hip). Sixteens are as decode attention.
//
// Few rows of a sequence (single tokens, what is left behind whole blocks) would leave most of
// a workgroup's waves idle: they are taken 16 at a time as decode attention takes its rows (by the
// steps of xp_attn_dev.h), every wave its own tiles from registers, and the waves join at the end.
//
// A batch is shared out on the device, from its lengths: every (block of rows or sixteen of
// rows, kv head) is a unit, and units with more tiles than an even share of the whole are cut
// along their positions, their pieces joined in order by a second launch.
//
// What bounds a block: of a tile's 4,530 cycles the matrix cores work 42%, the vector units 45%
// (a wave issues an exponential every 8.5 cycles, others every 5), both at once 14%, since the
// exponentials wait for the scores and the second product for them: 988 TFLOP/s, 2,048 rows of
// 32 heads of 128 behind 16,384 positions in 591 us. A mixed step of 512 rows and 16 single tokens
// behind up to 4,000 positions takes 67 us.
//
// Every workgroup forms the table of pieces for itself, 64 sequences a step and up to three times over
// the batch, before its first tile: little for tens of sequences, most of the time for many. 255
// single tokens behind up to 300 positions take 87 us and 1,000 of them 762 (32 heads of 128, 8 kv
// heads; their bytes take 11 and 42), behind up to 2,000 positions 159 and 1,199 (66 and 260).
#include "xp_attn_dev.h"

namespace xp {
namespace chunk {

using namespace attn;
using kv::Geo;

typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr float kLag = 2.0f, kBlockLift = 13.0f, kNear = 256.0f;   // as prompt attention's in fp16
constexpr int kWaves = 8;          // of a workgroup: two a SIMD, by registers
// Rows left behind whole blocks: up to kThin of them are taken by sixteens. Eight sequences of 64
// such rows behind up to 4,000 positions take 33 us as blocks and 39 as sixteens, 64 sequences of 32
// rows 113 and 96; one of 64 rows behind 30,000 40 and 34. At 256 columns 64 rows take 33 and 44.
// Where all sixteens have a workgroup each and contexts are up to kBrief tiles, all rows are taken
// by sixteens: a workgroup's waves then have the tiles at once (100 rows of 16 heads of 64 behind
// 200 positions: 6.9 us, as blocks 12.8).
constexpr int kThin = 32, kBrief = 16;

struct Item {
    int b, kind, first;        // sequence; block 0, sixteen 1; first row
    int piece, pieces, each;
    int slot;                  // of the unit's piece 0 at kv head 0, in pieces of its kind and all kv heads
};

struct Batch {
    Geo g;
    const uint16_t* q;
    long long q_stride;
    const uint8_t* cache;
    const int32_t* cu;
    const int32_t* start;
    const int32_t* table;
    uint16_t* out;
    long long out_stride;
    float* part[2];       // partial outputs of pieces of blocks and of sixteens, unscaled
    float* part_ml[2];    // their maxima, sums and the rows' factors
    Item* cuts;           // [0].b: how many units of a kv head are cut; then those
    int batch, rows, group, window;
    int thin;             // rows behind whole blocks up to which they are sixteens
    int share;            // workgroups that the batch is shared out to; 0: no unit is cut
    float scale_m;        // scale * log2(e) = scale_m * 2^scale_e
    int scale_e;
};

// What a wave of RW rows has of its products: RW x RW results, VE a lane, over KD of the
// contraction; lane (m, q) holds column m and, as element r, row at(r, q).
template <int RW>
struct Shape {
    static constexpr int VE = RW * RW / 64, KD = 512 / RW, NQ = 64 / RW;
    typedef __attribute__((ext_vector_type(VE))) float acc;
    static __device__ __forceinline__ int at(int r, int q) { return 4 * NQ * (r >> 2) + 4 * q + (r & 3); }
};
template <int RW>
__device__ __forceinline__ typename Shape<RW>::acc mma(h16x8 a, h16x8 b, typename Shape<RW>::acc c) {
    if constexpr (RW == 32)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Largest (or sum) over the lanes that share a row.
template <int RW, bool SUM>
__device__ __forceinline__ float over_q(float x) {
    const auto join = [](float a, float b) { return SUM ? a + b : fmaxf(a, b); };
    const uint32_t u = __float_as_uint(x);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = join(__uint_as_float(a[0]), __uint_as_float(a[1]));
    if constexpr (RW == 16) {
        const uint32_t w = __float_as_uint(x);
        const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
        x = join(__uint_as_float(b[0]), __uint_as_float(b[1]));
    }
    return x;
}

// LDS places, as prompt attention's. K: a row's 16-byte chunks are permuted so that 16
// neighbouring rows at one chunk index cover all banks; V: its blocks of RW columns.
template <int D>
__device__ __forceinline__ int k_at(int pos, int chunk) {
    const int s = D == 64 ? (pos >> 1) & 7 : pos & 15;
    return pos * (2 * D) + (chunk ^ s) * 16;
}
template <int D, int RW>
__device__ __forceinline__ int v_at(int pos, int block) {
    const int s = RW == 32 ? (D == 64 ? (pos >> 1) & 1 : pos & 3) : (D == 64 ? (pos >> 1) & 3 : pos & 7);
    return pos * (2 * D) + (block ^ s) * (2 * RW);
}
__device__ __forceinline__ h16x8 v_frag(const uint8_t* a, const uint8_t* b) {
    typedef __attribute__((ext_vector_type(8))) short s16x8;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)a);
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)b);
    return __builtin_bit_cast(h16x8, s16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
}
// Eight e2m1 codes times one scale, exact.
__device__ __forceinline__ h16x8 decode_by(uint32_t w, _Float16 s) {
    const h16x2 ss = h16x2{s, s};
    return decode8(w, ss, ss, ss, ss);
}

// Positions that a row sees: from lo to below hi, both within the table.
struct Span {
    int lo, hi;
};
__device__ __forceinline__ Span span_of(const Batch& a, long long at) {
    const long long cap = (long long)a.g.max_pages * a.g.page;
    const long long lo = a.window > 0 && at >= a.window ? at - a.window + 1 : 0;
    return Span{(int)(lo < cap ? lo : cap), (int)(at < 0 ? 0 : (at < cap ? at + 1 : cap))};
}

struct Seq {
    int q0, rows;         // first packed row; (token, head of a group) pairs
    long long start;
    int blocks, thin;     // whole blocks of rows (the last one may be a part); sixteens behind them
    int lo, tiles;        // first tile that a row sees, tiles up to the last one
};
template <int ROWS>
__device__ __forceinline__ Seq seq_of(const Batch& a, int b) {
    Seq s{};
    if (b >= a.batch) return s;
    s.q0 = a.cu[b];
    const long long n = (long long)a.cu[b + 1] - s.q0;
    if (s.q0 < 0 || n <= 0 || s.q0 + n > a.rows) return s;
    s.start = a.start[b];
    s.rows = (int)n * a.group;
    s.blocks = s.rows / ROWS;
    const int rest = s.rows - s.blocks * ROWS;
    s.blocks += rest > a.thin;
    s.thin = rest > a.thin ? 0 : (rest + 15) >> 4;
    const Span first = span_of(a, s.start), last = span_of(a, s.start + n - 1);
    s.lo = first.lo >> 6;
    const int hi = (last.hi + 63) >> 6;
    s.tiles = hi > s.lo ? hi - s.lo : 0;
    return s;
}

// How a unit is cut: pieces of `each` tiles, the last one what is left (none, if rounding has it so).
struct Cut {
    int pieces, each;
};
__device__ __forceinline__ Cut cut_of(int tiles, float limit) {
    if ((float)tiles <= limit) return Cut{1, tiles};
    const int p = (int)((float)(tiles - 1) / limit) + 1;
    return Cut{p, (int)((float)(tiles + p - 1) / (float)p)};
}

// Longest pieces, in tiles, of blocks and of sixteens: an even share of the work or more, so that
// there are at most twice as many pieces of cut units as workgroups that share it. A tile costs a
// block what kWaves tiles cost a sixteen, whose workgroup has that many at once (2.1 us); a piece
// kFixed of that and, when it is joined, kJoin.
// A join takes 9 us by itself, whence the shortest pieces.
constexpr float kLeast[2] = {8.0f, 16.0f};
constexpr float kFixed = 16.0f, kJoin = 0.15f;
// Up to so many sequences (a lane each) the best of 16 lengths is sought, beyond that pieces are an even
// share. Searched and even, 32 heads of 128: 512 rows and 15 single tokens behind up to 4,000 positions
// 77 and 86 us (in a graph), four pieces of up to 300 rows 77 and 100, 33 rows behind 65,000 69 and 86,
// 512 rows and 16 single tokens behind up to 30,000 347 and 418. Single tokens alone lose by it, the more
// of them: 8 behind up to 4,000 21 and 20, 32 47 and 41, 63 68 and 51; with a piece of 512 rows from some
// 24 on: 24 90 and 85, 32 86 and 87, 63 130 and 104: the estimate leaves their pieces longer than an even share.
constexpr int kSought = 64;
struct Limits {
    float tiles[2];
};
// Sum over the wave, in a fixed order.
__device__ __forceinline__ float wave_sum(float x) {
    const auto plus = [](float a, uint32_t b) { return a + __uint_as_float(b); };
    x = plus(x, dpp_or0<0x111, 0xF>(__float_as_uint(x)));
    x = plus(x, dpp_or0<0x112, 0xF>(__float_as_uint(x)));
    x = plus(x, dpp_or0<0x114, 0xF>(__float_as_uint(x)));
    x = plus(x, dpp_or0<0x118, 0xF>(__float_as_uint(x)));
    x = plus(x, dpp_or0<0x142, 0xA>(__float_as_uint(x)));
    x = plus(x, dpp_or0<0x143, 0xC>(__float_as_uint(x)));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
}
__device__ __forceinline__ Limits limits_by(float even, float grow) {
    return Limits{{fmaxf(kLeast[0], __builtin_ceilf(even * grow / kWaves)), fmaxf(kLeast[1], __builtin_ceilf(even * grow))}};
}
template <int ROWS>
__device__ __forceinline__ Limits limits_of(const Batch& a, const Seq& own) {
    const int lane = threadIdx.x & 63;
    if (!a.share) return Limits{{3e38f, 3e38f}};
    float all = 0.0f;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        const Seq s = b0 ? seq_of<ROWS>(a, b0 + lane) : own;
        all += wave_sum((float)(s.blocks * kWaves + s.thin) * (float)s.tiles);
    }
    // with room for the sums' rounding (1,024 of them at most): pieces are never shorter than an even share
    const float even = all * (float)a.g.kv_heads / (float)a.share * (1.0f + 0x1p-12f);
    if (a.batch > kSought) return limits_by(even, 1.0f);
    // Lanes 4 j .. 4 j + 3 try pieces of (1 + j^2 / 128) shares, the last four whole units, with a quarter of
    // the sequences each, and estimate when the workgroups that run at once are done: blocks in rounds,
    // sixteens in the gaps that they leave.
    const auto grow_of = [](int l) { return l >= 60 ? 1e30f : 1.0f + (float)((l >> 2) * (l >> 2)) / 128.0f; };
    const Limits l = limits_by(even, grow_of(lane));
    float n[2] = {0.0f, 0.0f}, work[2] = {0.0f, 0.0f}, most[2] = {0.0f, 0.0f}, joined = 0.0f;
    for (int b = 0; b < a.batch; b += 4) {
        const int at = b + (lane & 3);
        const float tiles = (float)__shfl(own.tiles, at);
        const float units[2] = {(float)__shfl(own.blocks, at), (float)__shfl(own.thin, at)};   // 0 behind the last sequence
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const float each = kind ? 1.0f : (float)kWaves;
            const float p = tiles > l.tiles[kind] ? __builtin_ceilf(tiles / l.tiles[kind]) : 1.0f;
            n[kind] += units[kind] * p;
            work[kind] += units[kind] * (each * tiles + kFixed * p);
            most[kind] = fmaxf(most[kind], units[kind] > 0.0f ? each * __builtin_ceilf(tiles / p) + kFixed : 0.0f);
            joined += p > 1.0f ? units[kind] * p * (kind ? 1.0f / 16.0f : 1.0f) : 0.0f;
        }
    }
#pragma unroll
    for (int i = 1; i <= 2; i <<= 1) {
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            n[kind] += __shfl_xor(n[kind], i);
            work[kind] += __shfl_xor(work[kind], i);
            most[kind] = fmaxf(most[kind], __shfl_xor(most[kind], i));
        }
        joined += __shfl_xor(joined, i);
    }
    const float kv = (float)a.g.kv_heads, at_once = (float)a.share;
    const float rounds = fmaxf(1.0f, __builtin_ceilf(n[0] * kv / at_once));
    float done = fminf(rounds * most[0], work[0] * kv / at_once + most[0]);
    const float left = work[1] * kv - (at_once * done - work[0] * kv);
    const float gaps = (at_once * rounds - n[0] * kv) * __builtin_floorf(done / fmaxf(most[1], 1.0f));
    if (left > 0.0f || n[1] * kv > gaps) done += fmaxf(left, 0.0f) / at_once + most[1];
    done = fmaxf(done, most[1]) + kJoin * joined * kv;
    const uint32_t best = wave_min_u32((done < 6e7f ? (uint32_t)done : 60000000u) << 6 | (uint32_t)lane);
    return limits_by(even, grow_of((int)(best & 63u)));
}

// Piece i of the launch, of all pieces of a kv head; false: there is none. Blocks come first,
// then sixteens; among up to 64 sequences those with the longest pieces, in four classes, so
// that short ones fill the gaps at the end; inside a sequence its last block, which sees most, is
// first. The workgroup that `lists` writes down the cut units of a kv head for the join.
template <int ROWS>
__device__ __forceinline__ bool find_item(const Batch& a, int i, bool lists, Item& it, Seq& sq) {
    const int lane = threadIdx.x & 63;
    const Seq own = seq_of<ROWS>(a, lane);
    const Limits limits = limits_of<ROWS>(a, own);
    int before = 0, listed = 0;
    bool found = false;
    for (int kind = 0; kind < 2; ++kind) {
        int cut_before = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 64) {
            const Seq s = b0 ? seq_of<ROWS>(a, b0 + lane) : own;
            const int units = kind ? s.thin : s.blocks;
            const Cut c = cut_of(s.tiles, kind ? limits.tiles[1] : limits.tiles[0]);
            const int items = units * c.pieces, slots = c.pieces > 1 ? items : 0;
            const int slot0 = cut_before + wave_incl_sum(slots) - slots;
            int first = 0;
            if (a.batch <= 64 && __popcll(__ballot(items > 0)) > 1) {
                const int top = (int)wave_max_u32((uint32_t)(items ? c.each : 0));
                const int part = (int)(4.0f * (float)c.each / (float)(top + 1)), cls = part > 3 ? 3 : part;
                for (int k = 3; k >= 0; --k) {
                    const int n = cls == k ? items : 0, incl = wave_incl_sum(n);
                    if (n) first = before + incl - n;
                    before += __builtin_amdgcn_readlane(incl, 63);
                }
            } else {
                const int incl = wave_incl_sum(items);
                first = before + incl - items;
                before += __builtin_amdgcn_readlane(incl, 63);
            }
            const auto first_row = [&](int blocks, int unit) { return kind ? blocks * ROWS + 16 * unit : unit * ROWS; };
            if (lists) {
                const int n = c.pieces > 1 ? units : 0, incl = wave_incl_sum(n);
                for (int u = 0; u < n; ++u)
                    a.cuts[1 + listed + incl - n + u] = Item{b0 + lane, kind, first_row(s.blocks, u), 0, c.pieces, c.each, slot0 + u * c.pieces};
                listed += __builtin_amdgcn_readlane(incl, 63);
            }
            const uint64_t hit = __ballot(items > 0 && first <= i && i - first < items);
            if (hit && !found) {
                const int l = __ffsll((unsigned long long)hit) - 1;
                const int rel = i - __builtin_amdgcn_readlane(first, l), n = __builtin_amdgcn_readlane(units, l);
                it.b = b0 + l;
                it.kind = kind;
                it.pieces = __builtin_amdgcn_readlane(c.pieces, l);
                it.each = __builtin_amdgcn_readlane(c.each, l);
                const int unit = n - 1 - rel / it.pieces;
                it.first = first_row(__builtin_amdgcn_readlane(s.blocks, l), unit);
                it.piece = rel % it.pieces;
                it.slot = __builtin_amdgcn_readlane(slot0, l) + unit * it.pieces;
                sq.q0 = __builtin_amdgcn_readlane(s.q0, l);
                sq.rows = __builtin_amdgcn_readlane(s.rows, l);
                sq.start = (long long)__builtin_amdgcn_readlane((int)(s.start >> 32), l) << 32 |
                           (long long)(uint32_t)__builtin_amdgcn_readlane((int)s.start, l);
                sq.lo = __builtin_amdgcn_readlane(s.lo, l);
                sq.tiles = __builtin_amdgcn_readlane(s.tiles, l);
                found = true;
                if (!lists) return true;
            }
            cut_before += __builtin_amdgcn_readlane(slot0 + slots, 63) - cut_before;
        }
    }
    if (lists && lane == 0) a.cuts[0].b = listed;
    return found;
}

// What the rows of a unit see: the first and last row's view, and the tiles of a piece.
struct View {
    Span first, last;
};
template <int ROWS>
__device__ __forceinline__ View view_of(const Batch& a, const Seq& s, const Item& it) {
    const int n = it.kind ? 16 : ROWS, last = (it.first + n < s.rows ? it.first + n : s.rows) - 1;
    return View{span_of(a, s.start + it.first / a.group), span_of(a, s.start + last / a.group)};
}
__device__ __forceinline__ Span tiles_of(const Seq& s, const View& v, const Item& it, int piece) {
    const int lo = v.first.lo >> 6, hi = (v.last.hi + 63) >> 6;
    const int p0 = s.lo + piece * it.each, p1 = piece + 1 < it.pieces ? p0 + it.each : s.lo + s.tiles;
    return Span{lo > p0 ? lo : p0, hi < p1 ? hi : p1};
}

// Partial outputs of a unit's piece: groups of RW rows (a block's waves, a sixteen is one), each
// RW * D / 256 kilobytes of four columns a lane, and the rows' maxima, sums and factors.
template <int D, int RW>
__device__ __forceinline__ f32x4* part_at(const Batch& a, int kind, long long group) {
    return (f32x4*)a.part[kind] + group * (RW * D / 4);
}

// 16 rows of a sequence: every wave takes its own tiles, as decode attention does.
template <int D, int ROWS, bool BF16>
__device__ __forceinline__ void thin_unit(const Batch& a, const Item& it, const Seq& sq, const View& view, int head, uint8_t* lds) {
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Span tl = tiles_of(sq, view, it, it.piece);
    const int row = it.first + c;
    const bool live = row < sq.rows;
    const int tok = live ? row / a.group : 0, hd = head * a.group + (live ? row - tok * a.group : 0);
    const Span sp = live ? span_of(a, sq.start + tok) : Span{0, 0};
    h16x8 qf[Dim<D>::NW];
    const float factor = row_frags<D, BF16>(a.q + (long long)(sq.q0 + tok) * a.q_stride + (long long)hd * D, live, q, a.scale_m, a.scale_e, qf);
    Running<D> r;
    r.clear();
    uint8_t* region = lds + wave * wave_v_bytes<D>();
    const int32_t* tr = a.table + (long long)it.b * a.g.max_pages;
    const int tiles = a.g.page >> 6;
    walk_tiles<D>(
        a.cache, tl.lo + wave, tl.hi, kWaves,
        [&](int tile, long long& place) {
            const int col = tile / tiles, id = tr[col];
            place = (((long long)id * a.g.kv_heads + head) * tiles + (tile - col * tiles)) * kv::tile_bytes(Dim<D>::NG);
            return (unsigned)id < (unsigned)a.g.n_pages ? tile : -1;
        },
        [&](int base, f32x4 (&s)[4], VTile<D>& v) {
            if (base >= view.last.lo && base + 64 <= view.first.hi) return false;
#pragma unroll
            for (int bl = 0; bl < 4; ++bl)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int pos = base + 16 * bl + 4 * q + e;
                    if (pos < sp.lo || pos >= sp.hi) s[bl][e] = -__builtin_inff();
                }
            return __ballot(clear_v<D>(v, view.last.hi - base, lane)) != 0;
        },
        [&](int base) { r.take_nan(region, sp.lo - base, sp.hi - base, q); }, qf, factor, r, region);
    const long long group = (long long)(it.slot + it.piece) * a.g.kv_heads + head;
    join_waves<D>(r, factor, lds, wave, kWaves, [&](int h, f32x4 o, float m, float l) {
        if (it.pieces > 1) {
            part_at<D, 16>(a, 1, group)[h * 64 + lane] = o;
            if (h == 0 && q == 0) {
                float* pm = a.part_ml[1] + group * 48 + c;
                pm[0] = m;
                pm[16] = l;
                pm[32] = factor;
            }
        } else if (live) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l; // nothing seen: zeros
            *(uint2*)(a.out + (long long)(sq.q0 + tok) * a.out_stride + (long long)hd * D + 16 * h + 4 * q) = to16<BF16>(o * inv);
        }
    });
}

// A block of rows, RW of them a wave, over tiles that all waves decode together.
template <int D, int RW, bool BF16>
__device__ __forceinline__ void block_unit(const Batch& a, const Item& it, const Seq& sq, const View& view, int head, uint8_t* lds) {
    typedef Shape<RW> Sh;
    typedef typename Sh::acc acc;
    constexpr int KD = Sh::KD, VE = Sh::VE, NG = D / 32;
    constexpr int NS = D / KD;                 // contraction steps of the scores
    constexpr int NT = 64 / RW;                // blocks of positions of the scores
    constexpr int ND = D / RW;                 // column blocks of the output
    constexpr int kTile = 64 * D * 2;          // bytes of a decoded tile of k, or of v
    constexpr int kUnits = 2 * NG;             // kilobytes of codes of a tile: NG of k, then NG of v
    constexpr int PER = (kUnits + kWaves - 1) / kWaves;   // a wave's
    constexpr int HB = 2 * NG;                 // 16-value columns of v
    uint32_t (*nan_v)[NG][2] = (uint32_t (*)[NG][2])(lds + 4 * kTile);   // [3]: positions of a tile whose values of a group are NaN and had to be taken out

    const int tid = threadIdx.x, lane = tid & 63, m = lane % RW, q = lane / RW;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Span tl = tiles_of(sq, view, it, it.piece);
    const Span sp_first = view.first, sp_last = view.last;

    const int row = it.first + wave * RW + m;
    const bool live = row < sq.rows;
    const bool busy = it.first + wave * RW < sq.rows;      // some row of the wave is
    const int tok = live ? row / a.group : 0;
    const int hd = head * a.group + (live ? row - tok * a.group : 0);
    const Span sp = live ? span_of(a, sq.start + tok) : Span{0, 0};
    const auto is_masked = [&](int tile) { return tile * 64 < sp_last.lo || tile * 64 + 64 > sp_first.hi; };

    h16x8 qf[NS];
    float factor, lag;
    {
        const uint16_t* qp = a.q + (long long)(sq.q0 + tok) * a.q_stride + (long long)hd * D + 8 * q;
        uint4 v[NS];
#pragma unroll
        for (int st = 0; st < NS; ++st) v[st] = live ? *(const uint4*)(qp + KD * st) : uint4{0, 0, 0, 0};
        int k = 0;
        if constexpr (BF16) {
            uint32_t top = 0;                  // exponent field of the row's largest magnitude
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                const uint32_t u[4] = {v[st].x, v[st].y, v[st].z, v[st].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = (u[i] >> 7) & 255u, hi = (u[i] >> 23) & 255u;
                    top = lo > top ? lo : top;
                    top = hi > top ? hi : top;
                }
            }
            const int e = (int)over_q<RW, false>((float)top);
            // largest magnitude to [2^14, 2^15); rows with an infinity or NaN are left as they are
            k = e == 255 ? 0 : 141 - e;
            k = k > 100 ? 100 : k;
            const float up = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                const uint32_t u[4] = {v[st].x, v[st].y, v[st].z, v[st].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qf[st][2 * i] = (_Float16)(__uint_as_float(u[i] << 16) * up);
                    qf[st][2 * i + 1] = (_Float16)(__uint_as_float(u[i] & 0xffff0000u) * up);
                }
            }
        } else {
#pragma unroll
            for (int st = 0; st < NS; ++st) qf[st] = __builtin_bit_cast(h16x8, v[st]);
        }
        // kept a normal number: a masked -inf times 0, or a score of 0 times infinity, would be NaN
        factor = fminf(fmaxf(__builtin_amdgcn_ldexpf(a.scale_m, a.scale_e - k), 0x1p-126f), 0x1p127f);
        lag = fminf(kLag / factor, 0x1p127f);              // finite: the maximum may be -infinity
    }

    // The next tile whose page exists (positions of others are not seen), tl.hi behind the last one,
    // and where its bytes are. A lane looks up one of 64 tiles, so that the page number of a tile is
    // not waited for (it took a fifth of the loop's time).
    const int32_t* tr = a.table + (long long)it.b * a.g.max_pages;
    const int page_tiles = a.g.page >> 6;
    int batch = tl.lo - 64, place_lo = 0, place_hi = 0;    // the first of the 64 tiles looked up
    uint64_t there = 0;                        // those of them that are left
    const auto find = [&](const uint8_t*& at) {
        while (!there) {
            batch += 64;
            if (batch >= tl.hi) {
                batch = tl.hi - 64;            // none then, however often it is asked
                return tl.hi;
            }
            const int own = batch + lane < tl.hi ? batch + lane : tl.hi - 1, col = own / page_tiles, id = tr[col];
            const long long place = (((long long)id * a.g.kv_heads + head) * page_tiles + (own - col * page_tiles)) * kv::tile_bytes(NG);
            place_lo = (int)place;
            place_hi = (int)(place >> 32);
            there = __ballot(batch + lane < tl.hi && (unsigned)id < (unsigned)a.g.n_pages);
        }
        const int l = __ffsll((unsigned long long)there) - 1;
        there &= there - 1;
        at = a.cache + ((long long)(uint32_t)__builtin_amdgcn_readlane(place_lo, l) | (long long)__builtin_amdgcn_readlane(place_hi, l) << 32);
        return batch + l;
    };
    // A wave's kilobytes of a tile: of k a group of all positions, a position a lane; of v
    // pairs of positions, neighbouring lanes at neighbouring columns, so that their decoded
    // pieces meet no bank twice.
    uint4 raw[PER];
    uint32_t scale[PER];
    const auto load = [&](const uint8_t* t) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int u = wave + j * kWaves;
            if (u < NG) {
                raw[j] = *(const uint4*)(t + u * 1024 + lane * 16);
                scale[j] = t[kv::k_scale(NG, lane, u)];
            } else if (u < kUnits) {
                const int h = lane % HB, pair = (u - NG) * (64 / HB) + lane / HB;
                raw[j] = *(const uint4*)(t + NG * 1088 + h * 512 + pair * 16);
                scale[j] = *(const uint16_t*)(t + kv::v_scale(NG, 2 * pair, h >> 1));
            }
        }
    };
    const auto stage = [&](int tile, uint8_t* lk, uint32_t (*nan)[2]) {
        uint8_t* lv = lk + kTile;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int u = wave + j * kWaves;
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            if (u < NG) {
                const h16x2 ss = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scale[j], 1.0f, false);
                const _Float16 s = ss.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) *(h16x8*)(lk + k_at<D>(lane, 4 * u + i)) = decode_by(w[i], s);
            } else if (u < kUnits) {
                const int h = lane % HB, pos = 2 * ((u - NG) * (64 / HB) + lane / HB);
                uint32_t sc = scale[j];
                if (is_masked(tile)) {
                    // Where not every row sees it: bytes behind the last row's position are no values,
                    // and a NaN scale must not meet the zero weight of a row that does not see it.
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool out = tile * 64 + pos + e >= sp_last.hi, odd = ((sc >> (8 * e)) & 127u) == 127u;
                        if (!out && odd) atomicOr(&nan[h >> 1][pos >> 5], 1u << ((pos + e) & 31));
                        if (out || odd) sc &= ~(255u << (8 * e));
                    }
                }
                const h16x2 s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc, 1.0f, false);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int to = RW == 32 ? v_at<D, RW>(pos + e, h >> 1) + (h & 1) * 32 : v_at<D, RW>(pos + e, h);
                        *(h16x8*)(lv + to + 16 * i) = decode_by(w[2 * e + i], e ? s.y : s.x);
                    }
            }
        }
    };

    acc o[ND], s[NT];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < VE; ++r) o[d][r] = 0.0f;
    float mx = -__builtin_inff(), sum = 0.0f;
    uint64_t far = 0;                          // lanes whose maximum is too large for one fma

    const auto form = [&](const uint8_t* lk) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < VE; ++r) s[i][r] = 0.0f;
#pragma unroll
        for (int st = 0; st < NS; ++st)
#pragma unroll
            for (int i = 0; i < NT; ++i)
                s[i] = mma<RW>(*(const h16x8*)(lk + k_at<D>(RW * i + m, KD / 8 * st + q)), qf[st], s[i]);
    };
    // What is not seen of a tile, and its maximum; returns what the exponentials' arguments start from.
    const auto settle = [&](int tile, const uint32_t (*nan)[2]) {
        if (is_masked(tile)) {
            const int here = tile * 64 + 4 * q;
#pragma unroll
            for (int e = 0; e < NT * VE; ++e) {
                const int ps = RW * (e / VE) + Sh::at(e % VE, 0) + here;
                if (ps >= sp.hi || ps < sp.lo) s[e / VE][e % VE] = -__builtin_inff();
            }
            // the NaN values that were taken out, for the rows that see them
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint64_t bad = (uint64_t)nan[g][1] << 32 | nan[g][0];
                if (!bad) continue;
                const int from = sp.lo - tile * 64, to = sp.hi - tile * 64;
                const uint64_t seen = (to >= 64 ? ~0ull : (to <= 0 ? 0ull : (1ull << to) - 1)) &
                                      (from <= 0 ? ~0ull : (from >= 64 ? 0ull : ~0ull << from));
                const float add = (bad & seen) ? __builtin_nanf("") : 0.0f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    if (d * RW / 32 == g)
#pragma unroll
                        for (int r = 0; r < VE; ++r) o[d][r] += add;
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int e = 1; e < NT * VE; ++e) top = fmaxf(top, s[e / VE][e % VE]);
        top = over_q<RW, false>(top);
        // Exponentials are taken from a maximum that lags behind; where it is too large for one
        // fma (a product with the factor, rounded, is within 2^-16 up to kNear), the factor
        // multiplies differences only, and nothing lags.
        if (__builtin_expect((__ballot(top > mx + lag) | far) != 0, 0)) {
            const float nm = fmaxf(top, mx), from = nm == -__builtin_inff() ? 0.0f : nm;
            const float alpha = __builtin_amdgcn_exp2f((mx - from) * factor);
            mx = nm;
            far = __ballot(!(__builtin_fabsf(from * factor) <= kNear));
            if (far)
#pragma unroll
                for (int e = 0; e < NT * VE; ++e) s[e / VE][e % VE] -= from;
            sum *= alpha;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] *= alpha;
        }
        return far || mx == -__builtin_inff() ? kBlockLift : __builtin_fmaf(-mx, factor, kBlockLift);
    };
    const auto add = [&](float base, const uint8_t* lv) {
        h16x8 p[NT * VE / 8];
#pragma unroll
        for (int e = 0; e < NT * VE; e += 2) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e / VE][e % VE], factor, base));
            const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[(e + 1) / VE][(e + 1) % VE], factor, base));
            const h16x2 xy = h16x2{(_Float16)x, (_Float16)y};
            p[e >> 3][e & 7] = xy.x;
            p[e >> 3][(e & 7) + 1] = xy.y;
            sum = __builtin_amdgcn_fdot2(xy, h16x2{(_Float16)1.0f, (_Float16)1.0f}, sum, false);
        }
        const int vrow = 4 * q + ((lane & 15) >> 2), vcol = (m >> 4) * 32 + (lane & 3) * 8;
#pragma unroll
        for (int st = 0; st < 64 / KD; ++st)
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const int pos = KD * st + vrow;
                o[d] = mma<RW>(v_frag(lv + v_at<D, RW>(pos, d) + vcol, lv + v_at<D, RW>(pos + KD / 2, d) + vcol), p[st], o[d]);
            }
    };

    const uint8_t* t = a.cache;
    int tile = find(t);
    if (tile < tl.hi) load(t);
    if (tid < 6 * NG) (&nan_v[0][0][0])[tid] = 0;
    __syncthreads();
    int next = tile < tl.hi ? find(t) : tl.hi;
    if (tile < tl.hi) stage(tile, lds, nan_v[0]);
    if (next < tl.hi) load(t);
    int n3 = 0;                                // this tile's place in nan_v
    for (int n = 0; tile < tl.hi; n ^= 1) {
        const int up = n3 == 2 ? 0 : n3 + 1;
        uint8_t* lk = lds + n * (2 * kTile);
        // the tile is in LDS, and everyone is done with the one before it
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        int after = tl.hi;
        if (next < tl.hi) {
            if (tid < 2 * NG) (&nan_v[n3 == 0 ? 2 : n3 - 1][0][0])[tid] = 0;
            stage(next, lds + (n ^ 1) * (2 * kTile), nan_v[up]);
            after = find(t);
            if (after < tl.hi) load(t);
        }
        if (busy) {
            form(lk);
            const float base = settle(tile, nan_v[n3]);
            add(base, lk + kTile);
        }
        tile = next;
        next = after;
        n3 = up;
    }

    sum = over_q<RW, true>(sum);
    if (it.pieces > 1) {
        if (!busy) return;
        const long long group = ((long long)(it.slot + it.piece) * a.g.kv_heads + head) * kWaves + wave;
        f32x4* po = part_at<D, RW>(a, 0, group) + lane;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int e = 0; e < VE; e += 4) po[(d * VE + e) / 4 * 64] = f32x4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]};
        if (q == 0) {
            float* pm = a.part_ml[0] + group * (3 * RW) + m;
            pm[0] = mx;
            pm[RW] = sum;
            pm[2 * RW] = factor;
        }
        return;
    }
    if (!live) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;     // nothing seen: zeros
    uint16_t* y = a.out + (long long)(sq.q0 + tok) * a.out_stride + (long long)hd * D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < VE; e += 4)
            *(uint2*)(y + RW * d + Sh::at(e, q)) = to16<BF16>(f32x4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]} * inv);
}

template <int D>
constexpr int block_rows() {
    return D == 256 ? 128 : 256;
}
template <int D>
constexpr int lds_bytes() {
    constexpr int block = 4 * 64 * D * 2 + 3 * (D / 32) * 8, thin = kWaves * wave_join_bytes<D>();
    static_assert(wave_join_bytes<D>() >= wave_v_bytes<D>());
    return block > thin ? block : thin;
}

template <int D, bool BF16>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_chunk_kernel(Batch a) {
    constexpr int ROWS = block_rows<D>();
    __shared__ __attribute__((aligned(16))) uint8_t lds[lds_bytes<D>()];
    const int head = blockIdx.x % a.g.kv_heads;
    Item it;
    Seq sq{};
    if (!find_item<ROWS>(a, blockIdx.x / a.g.kv_heads, a.share && blockIdx.x == gridDim.x - 1 && __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) == 0, it, sq))
        return;
    // the same in all lanes, which the compiler does not see by itself
    const auto same = [](int& x) { x = __builtin_amdgcn_readfirstlane(x); };
    for (int* x : {&it.b, &it.kind, &it.first, &it.piece, &it.pieces, &it.each, &it.slot, &sq.q0, &sq.rows, &sq.lo, &sq.tiles}) same(*x);
    sq.start = (long long)__builtin_amdgcn_readfirstlane((int)(sq.start >> 32)) << 32 |
               (long long)(uint32_t)__builtin_amdgcn_readfirstlane((int)sq.start);
    const View view = view_of<ROWS>(a, sq, it);
    const Span tl = tiles_of(sq, view, it, it.piece);
    if (it.pieces > 1 && tl.lo >= tl.hi) return;           // the join knows
    if (it.kind)
        thin_unit<D, ROWS, BF16>(a, it, sq, view, head, lds);
    else
        block_unit<D, ROWS / kWaves, BF16>(a, it, sq, view, head, lds);
}

// Joins the pieces of a cut unit, in order: a workgroup takes four of the kilobytes of a group of
// rows, its waves take the pieces in turn, and meet in LDS.
constexpr int kJoinWaves = 4, kJoinParts = 4;
template <int D, int RW, bool BF16>
__device__ __forceinline__ void join_group(const Batch& a, const Item& it, const Seq& sq, int head, int p0, int p1, int groups, int g, int part,
                                           f32x4 (*so)[kJoinParts][64], float (*sml)[2][64]) {
    constexpr int VE = Shape<RW>::VE;
    const int lane = threadIdx.x & 63, m = lane % RW, q = lane / RW, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const auto at = [&](int piece) { return ((long long)(it.slot + piece) * a.g.kv_heads + head) * groups + g; };
    // the row's, the same with every piece
    const float factor = p0 < p1 ? a.part_ml[it.kind][at(p0) * (3 * RW) + 2 * RW + m] : 1.0f;
    float mx = -__builtin_inff(), sum = 0.0f;
    f32x4 o[kJoinParts];
#pragma unroll
    for (int j = 0; j < kJoinParts; ++j) o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int U = 4;
    for (int s = p0 + wave; s < p1; s += U * kJoinWaves) {
        f32x4 v[U][kJoinParts];
        float vm[U], vl[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long from = at(s + u * kJoinWaves < p1 ? s + u * kJoinWaves : s);
            vm[u] = a.part_ml[it.kind][from * (3 * RW) + m];
            vl[u] = a.part_ml[it.kind][from * (3 * RW) + RW + m];
#pragma unroll
            for (int j = 0; j < kJoinParts; ++j) v[u][j] = part_at<D, RW>(a, it.kind, from)[(part + j) * 64 + lane];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u * kJoinWaves >= p1) break;
            const float nm = fmaxf(mx, vm[u]), from = nm == -__builtin_inff() ? 0.0f : nm;
            const float fa = __builtin_amdgcn_exp2f((mx - from) * factor), fb = __builtin_amdgcn_exp2f((vm[u] - from) * factor);
            mx = nm;
            sum = sum * fa + vl[u] * fb;
#pragma unroll
            for (int j = 0; j < kJoinParts; ++j) o[j] = o[j] * fa + v[u][j] * fb;
        }
    }
#pragma unroll
    for (int j = 0; j < kJoinParts; ++j) so[wave][j][lane] = o[j];
    sml[wave][0][lane] = mx;
    sml[wave][1][lane] = sum;
    __syncthreads();
    const int row = it.first + g * RW + m;
    if (row >= sq.rows) return;
    float jm = -__builtin_inff(), jl = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) jm = fmaxf(jm, sml[w][0][lane]);
    const float from = jm == -__builtin_inff() ? 0.0f : jm;
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f((sml[w][0][lane] - from) * factor);
        jl = __builtin_fmaf(sml[w][1][lane], f, jl);
        acc += so[w][wave][lane] * f;          // wave w ends with kilobyte w
    }
    part += wave;
    const int tok = row / a.group, hd = head * a.group + row - tok * a.group;
    const float inv = jl == 0.0f ? 0.0f : 1.0f / jl;
    *(uint2*)(a.out + (long long)(sq.q0 + tok) * a.out_stride + (long long)hd * D + RW * (part / (VE / 4)) +
              Shape<RW>::at(part % (VE / 4) * 4, q)) = to16<BF16>(acc * inv);
}
template <int D, bool BF16>
__global__ __launch_bounds__(64 * kJoinWaves) void chunk_join_kernel(Batch a) {
    constexpr int ROWS = block_rows<D>(), RW = ROWS / kWaves, kParts = RW * D / 256;
    static_assert(kJoinWaves == kJoinParts && kParts % kJoinParts == 0 && D / 16 % kJoinParts == 0);
    __shared__ f32x4 so[kJoinWaves][kJoinParts][64];
    __shared__ float sml[kJoinWaves][2][64];
    const int head = blockIdx.y % a.g.kv_heads, unit = blockIdx.y / a.g.kv_heads, part = blockIdx.x * kJoinParts;
    if (unit >= a.cuts[0].b) return;
    const Item it = a.cuts[1 + unit];
    if (it.kind && part >= D / 16) return;
    const Seq sq = seq_of<ROWS>(a, it.b);
    const int g = part / kParts;
    if (it.kind == 0 && it.first + g * RW >= sq.rows) return;
    const View view = view_of<ROWS>(a, sq, it);
    // the pieces in which the unit has tiles: one after the other
    int p0 = 0, p1 = it.pieces;
    const auto empty = [&](int p) {
        const Span t = tiles_of(sq, view, it, p);
        return t.lo >= t.hi;
    };
    while (p0 < p1 - 1 && empty(p0)) ++p0;
    while (p1 > p0 + 1 && empty(p1 - 1)) --p1;
    if (empty(p0)) p1 = p0;                    // a unit that sees nothing
    if (it.kind)
        join_group<D, 16, BF16>(a, it, sq, head, p0, p1, 1, 0, part, so, sml);
    else
        join_group<D, RW, BF16>(a, it, sq, head, p0, p1, kWaves, g, part % kParts, so, sml);
}

constexpr int kCus = 256;

struct Launch {
    long long units;               // at most
    int thin;
    int share, cut;                // workgroups of an even share; units that are cut at most
    size_t part[2], ml[2], total;
};
static Launch plan_of(const xp_kv_dims* d, int heads, int rows, int batch, int max_len) {
    Launch p{};
    const long long pairs = (long long)rows * (heads / d->kv_heads), each = d->head_dim == 256 ? 128 : 256;
    const int tiles = (int)(((long long)max_len + 63) / 64);
    // whole blocks, and behind them of every sequence a part of one or up to thin / 16 sixteens
    const long long rest = pairs / 16 + batch;
    p.thin = tiles <= kBrief && rest * d->kv_heads <= kCus ? (int)each : kThin;
    const long long most = (long long)batch * (p.thin / 16);
    p.units = (pairs / each + (rest < most ? rest : most)) * d->kv_heads;
    // A piece saves 0.4 us for every 8 tiles that it takes off a sixteen, 2.2 us for each that it takes off a
    // block, and a join takes 9 us: where all rows are sixteens it pays for longer sequences only.
    p.share = tiles > (pairs > p.thin ? 8 : 32) ? kCus : 0;
    p.cut = (int)(p.units < p.share ? p.units : p.share);
    size_t at = p.share ? align256((p.share + 1) * sizeof(Item)) : 0;
    for (int kind = 0; kind < 2; ++kind) {
        const size_t held = (size_t)(2 * p.share) * (kind ? 16 : each);
        p.part[kind] = at;
        at += held * d->head_dim * sizeof(float);
        p.ml[kind] = at;
        at += held * 3 * sizeof(float);
    }
    p.total = at ? at : 16;
    return p;
}

static int check_chunk(const xp_kv_dims* d, int heads, int batch, int max_pages, int rows, int max_len) {
    const int st = kv::check_geo(d, batch, max_pages);
    if (st != XP_OK) return st;
    if (heads < 1 || heads > 65535 || heads % d->kv_heads || rows < 0 || max_len < 0) return XP_ERR_SHAPE;
    const long long pairs = (long long)rows * (heads / d->kv_heads);
    if (pairs > 0x7fffffff - 256) return XP_ERR_SHAPE;
    const Launch p = plan_of(d, heads, rows, batch, max_len);
    // workgroups of 512 threads: a launch has fewer than 2^32
    return p.units + p.share + d->kv_heads >= (1 << 23) ? XP_ERR_SHAPE : XP_OK;
}

template <int D, bool BF16>
static int launch(const Batch& a, const Launch& p, hipStream_t s) {
    const unsigned kv = (unsigned)a.g.kv_heads;
    const auto all_heads = [&](int n) { return ((unsigned)n + kv - 1) / kv * kv; };
    hipLaunchKernelGGL((attn_chunk_kernel<D, BF16>), dim3((unsigned)p.units + all_heads(p.share)), dim3(64 * kWaves), 0, s, a);
    // a block's kilobytes; a sixteen's are fewer
    constexpr int kParts = block_rows<D>() * D / 256 / kJoinParts;
    if (p.share) hipLaunchKernelGGL((chunk_join_kernel<D, BF16>), dim3(kParts, all_heads(p.cut)), dim3(64 * kJoinWaves), 0, s, a);
    return launch_status();
}

}  // namespace chunk
}  // namespace xp

using namespace xp;
using namespace xp::chunk;

XP_API size_t xp_attn_chunk_workspace_bytes(const xp_kv_dims* dims, int32_t heads, int32_t rows, int32_t batch, int32_t max_len) {
    if (check_chunk(dims, heads, batch, 1, rows, max_len) != XP_OK) return 0;
    return plan_of(dims, heads, rows, batch, max_len).total;
}

XP_API int xp_attn_chunk(const xp_kv_dims* dims, int32_t heads, int32_t batch, int32_t max_pages, int32_t rows, int32_t max_len,
                         int32_t type, const void* q, int64_t q_stride, float scale, int32_t window, const uint8_t* cache,
                         const int32_t* table, const int32_t* cu_rows, const int32_t* start, void* out, int64_t out_stride,
                         void* workspace, size_t ws_bytes, void* stream) {
    const int st = check_chunk(dims, heads, batch, max_pages, rows, max_len);
    if (st != XP_OK) return st;
    if ((type != XP_BF16 && type != XP_F16) || window < 0 || !(scale > 0.0f && scale < __builtin_inff())) return XP_ERR_SHAPE;
    if (batch == 0 || rows == 0) return XP_OK;
    if (!q || !cache || !table || !cu_rows || !start || !out || !workspace) return XP_ERR_NULL;
    const int64_t width = (int64_t)heads * dims->head_dim;
    if (q_stride < width || out_stride < width || q_stride % 8 || out_stride % 4 || !kv::aligned_to(q, 16) ||
        !kv::aligned_to(out, 8) || !kv::aligned_to(cache, 16) || !kv::aligned_to(table, 4) || !kv::aligned_to(cu_rows, 4) ||
        !kv::aligned_to(start, 4) || !kv::aligned_to(workspace, 16))
        return XP_ERR_SHAPE;
    // a workgroup's q is read before its rows are written; pieces of a unit write to the workspace only
    const kv::Rows qr{q, rows, 2 * q_stride, 2 * width}, yr{out, rows, 2 * out_stride, 2 * width};
    if (!qr.same(yr) && kv::rows_meet(qr, yr)) return XP_ERR_SHAPE;
    const Launch p = plan_of(dims, heads, rows, batch, max_len);
    // every workgroup forms the table of pieces from cu and start: were these written over, tables would differ
    // and pieces lie anywhere
    const kv::Rows read[] = {kv::flat(cache, (int64_t)xp_kv_bytes(dims)), kv::flat(table, 4 * (int64_t)batch * max_pages),
                             kv::flat(cu_rows, 4 * (int64_t)batch + 4), kv::flat(start, 4 * (int64_t)batch), qr, yr};
    if (kv::meets_any(yr, read, 4)) return XP_ERR_SHAPE;
    if (p.share && kv::meets_any(kv::flat(workspace, (int64_t)(ws_bytes < p.total ? ws_bytes : p.total)), read, 6)) return XP_ERR_SHAPE;
    if (ws_bytes < p.total) return XP_ERR_WORKSPACE;
    Batch a{};
    a.g = kv::geo_of(dims, max_pages);
    a.q = (const uint16_t*)q;
    a.q_stride = q_stride;
    a.cache = cache;
    a.cu = cu_rows;
    a.start = start;
    a.table = table;
    a.out = (uint16_t*)out;
    a.out_stride = out_stride;
    a.cuts = (Item*)workspace;
    for (int kind = 0; kind < 2; ++kind) {
        a.part[kind] = (float*)((char*)workspace + p.part[kind]);
        a.part_ml[kind] = (float*)((char*)workspace + p.ml[kind]);
    }
    a.batch = batch;
    a.rows = rows;
    a.group = heads / dims->kv_heads;
    a.window = window;
    a.thin = p.thin;
    a.share = p.share;
    a.scale_m = (float)__builtin_frexp((double)scale * 1.4426950408889634, &a.scale_e);
    hipStream_t s = (hipStream_t)stream;
    const bool bf = type == XP_BF16;
    switch (dims->head_dim) {
        case 64: return bf ? launch<64, true>(a, p, s) : launch<64, false>(a, p, s);
        case 128: return bf ? launch<128, true>(a, p, s) : launch<128, false>(a, p, s);
        default: return bf ? launch<256, true>(a, p, s) : launch<256, false>(a, p, s);
    }
}
