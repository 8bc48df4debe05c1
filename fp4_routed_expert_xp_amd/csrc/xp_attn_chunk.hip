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
// ones; the maximum may lag by 2^2 (see xp_attn_prompt.hip).
//
// A batch is shared out on the device, from its lengths: every (block of rows, kv head) is
// a unit, and sequences with more tiles than an even share of the whole are cut along
// their positions, their pieces joined in order by a second launch.
#include "xp_kv_dev.h"

namespace xp {
namespace chunk {

using kv::Geo;

typedef __attribute__((ext_vector_type(2))) _Float16 h16x2;
typedef __attribute__((ext_vector_type(8))) _Float16 h16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr float kLag = 2.0f, kLift = 13.0f, kNear = 256.0f;   // as prompt attention's in fp16

struct Args {
    Geo g;
    const uint16_t* q;
    long long q_stride;
    const uint8_t* cache;
    const int32_t* cu;
    const int32_t* start;
    const int32_t* table;
    uint16_t* out;
    long long out_stride;
    float* part;          // partial outputs of pieces, unscaled
    float* part_ml;       // their maxima, sums and the rows' factors
    int batch, rows, group, window;
    int share, least;     // sequences longer than max(tiles of all units / share, least) tiles are cut; share 0: none
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
// Eight e2m1 codes times their scale, exact.
__device__ __forceinline__ h16x8 decode8(uint32_t w, _Float16 s) {
    const h16x2 ss = h16x2{s, s};
    const h16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * ss, b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * ss;
    const h16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * ss, d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * ss;
    return h16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
// Four results to 16 bits, nearest even.
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

// Positions that a row sees: from lo to below hi, both within the table.
struct Span {
    int lo, hi;
};
__device__ __forceinline__ Span span_of(const Args& a, long long at) {
    const long long cap = (long long)a.g.max_pages * a.g.page;
    const long long lo = a.window > 0 && at >= a.window ? at - a.window + 1 : 0;
    return Span{(int)(lo < cap ? lo : cap), (int)(at < 0 ? 0 : (at < cap ? at + 1 : cap))};
}

struct Seq {
    int q0, rows;         // first packed row; (token, head of a group) pairs
    long long start;
    int blocks, lo, tiles;   // blocks of rows; first tile that a row sees, tiles up to the last one
};
template <int ROWS>
__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
    Seq s{0, 0, 0, 0, 0, 0};
    if (b >= a.batch) return s;
    s.q0 = a.cu[b];
    const long long n = (long long)a.cu[b + 1] - s.q0;
    if (s.q0 < 0 || n <= 0 || s.q0 + n > a.rows) return s;
    s.start = a.start[b];
    s.rows = (int)n * a.group;
    s.blocks = (s.rows + ROWS - 1) / ROWS;
    const Span first = span_of(a, s.start), last = span_of(a, s.start + n - 1);
    s.lo = first.lo >> 6;
    const int hi = (last.hi + 63) >> 6;
    s.tiles = hi > s.lo ? hi - s.lo : 0;
    return s;
}

// How a sequence is cut: pieces of `each` tiles.
struct Cut {
    int pieces, each;
};
__device__ __forceinline__ Cut cut_of(int tiles, int limit) {
    const int p = tiles > limit ? (tiles - 1) / limit + 1 : 1;
    return Cut{p, (tiles + p - 1) / p};
}
__device__ __forceinline__ long long wave_sum(long long x) {
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) x += __shfl_xor(x, i);
    return x;
}

struct Item {
    int b, block, piece, pieces, each, slot;   // slot: of the unit's piece 0 at kv head 0, in pieces of all kv heads
};
// Piece i of the launch, of all pieces of a kv head (JOIN: cut unit i); false: there is
// none. Among up to 64 sequences those with the longest pieces come first, in four classes,
// so that short ones fill the gaps at the end; inside a sequence its last block, which sees
// most, is first.
template <int ROWS, bool JOIN>
__device__ __forceinline__ bool find_item(const Args& a, int i, Item& it) {
    const int lane = threadIdx.x & 63;
    int limit = 0x7fffffff;
    if (a.share) {
        long long all = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 64) {
            const Seq s = seq_of<ROWS>(a, b0 + lane);
            all += (long long)s.blocks * s.tiles;
        }
        all = wave_sum(all) * a.g.kv_heads;
        const long long even = (all + a.share - 1) / a.share;
        limit = even < a.least ? a.least : (even > (1 << 26) ? 1 << 26 : (int)even);
    }
    int before = 0, cut_before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        const Seq s = seq_of<ROWS>(a, b0 + lane);
        const Cut c = cut_of(s.tiles, limit);
        const bool cut = s.blocks > 0 && c.pieces > 1;
        const int items = JOIN ? (cut ? s.blocks : 0) : s.blocks * c.pieces, slots = cut ? s.blocks * c.pieces : 0;
        int first = 0;
        if (!JOIN && a.batch <= 64) {
            const int top = (int)wave_max_u32((uint32_t)(items ? c.each : 0));
            const int cls = (int)(4.0f * (float)c.each / (float)(top + 1));
            for (int k = 3; k >= 0; --k) {
                const int n = (cls > 3 ? 3 : cls) == k ? items : 0, incl = wave_incl_sum(n);
                if (n) first = before + incl - n;
                before += __builtin_amdgcn_readlane(incl, 63);
            }
        } else {
            const int incl = wave_incl_sum(items);
            first = before + incl - items;
            before += __builtin_amdgcn_readlane(incl, 63);
        }
        const int cut_incl = wave_incl_sum(slots);
        const uint64_t hit = __ballot(items > 0 && first <= i && i - first < items);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            const int rel = i - __builtin_amdgcn_readlane(first, l), blocks = __builtin_amdgcn_readlane(s.blocks, l);
            it.b = b0 + l;
            it.pieces = __builtin_amdgcn_readlane(c.pieces, l);
            it.each = __builtin_amdgcn_readlane(c.each, l);
            it.block = JOIN ? rel : blocks - 1 - rel / it.pieces;
            it.piece = JOIN ? 0 : rel % it.pieces;
            it.slot = cut_before + __builtin_amdgcn_readlane(cut_incl - slots, l) + it.block * it.pieces;
            return true;
        }
        cut_before += __builtin_amdgcn_readlane(cut_incl, 63);
    }
    return false;
}

// A block's tiles within its sequence's piece: [lo, hi).
template <int ROWS>
__device__ __forceinline__ Span tiles_of(const Args& a, const Seq& s, const Item& it, int piece) {
    const int first = it.block * ROWS, last = (first + ROWS < s.rows ? first + ROWS : s.rows) - 1;
    const int lo = span_of(a, s.start + first / a.group).lo >> 6, hi = (span_of(a, s.start + last / a.group).hi + 63) >> 6;
    const int p0 = s.lo + piece * it.each, p1 = piece + 1 < it.pieces ? p0 + it.each : s.lo + s.tiles;
    return Span{lo > p0 ? lo : p0, hi < p1 ? hi : p1};
}

template <int D, int RW, int WAVES, bool BF16>
__global__ __launch_bounds__(64 * WAVES, 2) void attn_chunk_kernel(Args a) {
    typedef Shape<RW> Sh;
    typedef typename Sh::acc acc;
    constexpr int KD = Sh::KD, VE = Sh::VE, ROWS = RW * WAVES, NG = D / 32;
    constexpr int NS = D / KD;                 // contraction steps of the scores
    constexpr int NT = 64 / RW;                // blocks of positions of the scores
    constexpr int ND = D / RW;                 // column blocks of the output
    constexpr int kTile = 64 * D * 2;          // bytes of a decoded tile of k, or of v
    constexpr int kUnits = 2 * NG;             // kilobytes of codes of a tile: NG of k, then NG of v
    constexpr int PER = (kUnits + WAVES - 1) / WAVES;   // a wave's
    constexpr int HB = 2 * NG;                 // 16-value columns of v
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][2 * kTile];
    __shared__ uint32_t nan_v[3][NG][2];       // positions of a tile whose values of a group are NaN and had to be taken out

    const int tid = threadIdx.x, lane = tid & 63, m = lane % RW, q = lane / RW;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int head = blockIdx.x % a.g.kv_heads;
    Item it;
    if (!find_item<ROWS, false>(a, blockIdx.x / a.g.kv_heads, it)) return;
    const Seq sq = seq_of<ROWS>(a, it.b);
    const Span tl = tiles_of<ROWS>(a, sq, it, it.piece);
    if (it.pieces > 1 && tl.lo >= tl.hi) return;           // the join knows

    const int row = it.block * ROWS + wave * RW + m;
    const bool live = row < sq.rows;
    const bool busy = it.block * ROWS + wave * RW < sq.rows;   // some row of the wave is
    const int tok = live ? row / a.group : 0;
    const int hd = head * a.group + (live ? row - tok * a.group : 0);
    const Span sp = live ? span_of(a, sq.start + tok) : Span{0, 0};
    // what all of the workgroup's rows see, and where its last row's view ends
    const int first_row = it.block * ROWS, last_row = (first_row + ROWS < sq.rows ? first_row + ROWS : sq.rows) - 1;
    const Span sp_first = span_of(a, sq.start + first_row / a.group), sp_last = span_of(a, sq.start + last_row / a.group);
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

    // The next tile at or behind `tile` whose page exists (positions of others are not
    // seen), and where its bytes are; page column and place on the page follow it.
    const int32_t* tr = a.table + (long long)it.b * a.g.max_pages;
    const int page_tiles = a.g.page >> 6;
    int col = tl.lo / page_tiles, in_page = tl.lo - col * page_tiles;
    const auto find = [&](int& tile) {
        for (; tile < tl.hi; ++tile) {
            const int id = tr[col];
            const long long at = (((long long)id * a.g.kv_heads + head) * page_tiles + in_page) * kv::tile_bytes(NG);
            if (++in_page == page_tiles) {
                in_page = 0;
                ++col;
            }
            if ((unsigned)id < (unsigned)a.g.n_pages) return a.cache + at;
        }
        return a.cache;
    };
    // A wave's kilobytes of a tile: of k a group of all positions, a position a lane; of v
    // pairs of positions, neighbouring lanes at neighbouring columns, so that their decoded
    // pieces meet no bank twice.
    uint4 raw[PER];
    uint32_t scale[PER];
    const auto load = [&](const uint8_t* t) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int u = wave + j * WAVES;
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
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int u = wave + j * WAVES;
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            if (u < NG) {
                const h16x2 ss = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scale[j], 1.0f, false);
                const _Float16 s = ss.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) *(h16x8*)(lk + k_at<D>(lane, 4 * u + i)) = decode8(w[i], s);
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
                uint8_t* lv = lk + kTile;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int to = RW == 32 ? v_at<D, RW>(pos + e, h >> 1) + (h & 1) * 32 : v_at<D, RW>(pos + e, h);
                        *(h16x8*)(lv + to + 16 * i) = decode8(w[2 * e + i], e ? s.y : s.x);
                    }
            }
        }
    };

    acc o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < VE; ++r) o[d][r] = 0.0f;
    float mx = -__builtin_inff(), sum = 0.0f;
    uint64_t far = 0;                          // lanes whose maximum is too large for one fma

    int tile = tl.lo;
    const uint8_t* t = find(tile);
    if (tile < tl.hi) load(t);
    if (tid < 6 * NG) (&nan_v[0][0][0])[tid] = 0;
    __syncthreads();
    int next = tile + 1;
    const uint8_t* nt = find(next);
    if (tile < tl.hi) stage(tile, lds[0], nan_v[0]);
    if (next < tl.hi) load(nt);

    for (int turn = 0, clear = 0; tile < tl.hi; turn ^= 1, clear = clear == 2 ? 0 : clear + 1) {
        uint8_t* lk = lds[turn];
        uint8_t* lv = lk + kTile;
        uint32_t (*nan)[2] = nan_v[clear];
        // the tile is in LDS, and everyone is done with the one before it
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        int after = next + 1;
        if (next < tl.hi) {
            if (tid < 2 * NG) (&nan_v[clear == 0 ? 2 : clear - 1][0][0])[tid] = 0;
            stage(next, lds[turn ^ 1], nan_v[clear == 2 ? 0 : clear + 1]);
            const uint8_t* at = find(after);
            if (after < tl.hi) load(at);
        }
        const bool masked = is_masked(tile);
        if (busy) {
            acc s[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int r = 0; r < VE; ++r) s[i][r] = 0.0f;
#pragma unroll
            for (int st = 0; st < NS; ++st)
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    s[i] = mma<RW>(*(const h16x8*)(lk + k_at<D>(RW * i + m, KD / 8 * st + q)), qf[st], s[i]);
            if (masked) {
                const int here = tile * 64 + 4 * q;
#pragma unroll
                for (int e = 0; e < NT * VE; ++e) {
                    const int ps = RW * (e / VE) + Sh::at(e % VE, 0) + here;
                    if (ps >= sp.hi || ps < sp.lo) s[e / VE][e % VE] = -__builtin_inff();
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
            const float base = far || mx == -__builtin_inff() ? kLift : __builtin_fmaf(-mx, factor, kLift);
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
            if (masked) {
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
            const int vrow = 4 * q + ((lane & 15) >> 2), vcol = (m >> 4) * 32 + (lane & 3) * 8;
#pragma unroll
            for (int st = 0; st < 64 / KD; ++st)
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const int pos = KD * st + vrow;
                    o[d] = mma<RW>(v_frag(lv + v_at<D, RW>(pos, d) + vcol, lv + v_at<D, RW>(pos + KD / 2, d) + vcol), p[st], o[d]);
                }
        }
        tile = next;
        next = after;
    }

    sum = over_q<RW, true>(sum);
    if (it.pieces > 1) {
        if (!busy) return;
        const long long slot = (long long)(it.slot + it.piece) * a.g.kv_heads + head;
        f32x4* po = (f32x4*)a.part + (slot * WAVES + wave) * (ND * VE / 4 * 64) + lane;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int e = 0; e < VE; e += 4) po[(d * VE + e) / 4 * 64] = f32x4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]};
        if (q == 0) {
            float* pm = a.part_ml + (slot * WAVES + wave) * (3 * RW) + m;
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

// Joins the pieces of a cut unit, in order: a workgroup for the rows of one wave, whose
// partial outputs its own waves share out as kilobytes.
template <int D, int RW, int WAVES, bool BF16>
__global__ __launch_bounds__(256) void chunk_join_kernel(Args a) {
    constexpr int VE = Shape<RW>::VE, ROWS = RW * WAVES, ND = D / RW, kParts = ND * VE / 4;
    const int lane = threadIdx.x & 63, m = lane % RW, q = lane / RW, wave = blockIdx.x;
    const int head = blockIdx.y % a.g.kv_heads;
    Item it;
    if (!find_item<ROWS, true>(a, blockIdx.y / a.g.kv_heads, it)) return;
    const Seq sq = seq_of<ROWS>(a, it.b);
    const int row = it.block * ROWS + wave * RW + m;
    if (it.block * ROWS + wave * RW >= sq.rows) return;
    const bool live = row < sq.rows;
    const int tok = live ? row / a.group : 0;
    const int hd = head * a.group + (live ? row - tok * a.group : 0);
    const auto slot = [&](int piece) { return ((long long)(it.slot + piece) * a.g.kv_heads + head) * WAVES + wave; };
    // the pieces in which the block has tiles: one after the other
    int p0 = 0, p1 = it.pieces;
    while (p0 < p1 && tiles_of<ROWS>(a, sq, it, p0).lo >= tiles_of<ROWS>(a, sq, it, p0).hi) ++p0;
    while (p1 > p0 && tiles_of<ROWS>(a, sq, it, p1 - 1).lo >= tiles_of<ROWS>(a, sq, it, p1 - 1).hi) --p1;
    float mx = -__builtin_inff(), sum = 0.0f, factor = 0.0f;
    for (int p = p0; p < p1; ++p) mx = fmaxf(mx, a.part_ml[slot(p) * (3 * RW) + m]);
    const float from = mx == -__builtin_inff() ? 0.0f : mx;
    f32x4 o[(kParts + 3) / 4];
#pragma unroll
    for (int j = 0; j < (kParts + 3) / 4; ++j) o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int p = p0; p < p1; ++p) {
        const float* pm = a.part_ml + slot(p) * (3 * RW) + m;
        factor = pm[2 * RW];
        const float f = __builtin_amdgcn_exp2f((pm[0] - from) * factor);
        sum = __builtin_fmaf(pm[RW], f, sum);
        const f32x4* po = (const f32x4*)a.part + slot(p) * (kParts * 64) + lane;
#pragma unroll
        for (int j = 0; j < (kParts + 3) / 4; ++j) {
            const int part = (threadIdx.x >> 6) + 4 * j;
            if (part < kParts) o[j] += po[part * 64] * f;
        }
    }
    if (!live) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t* y = a.out + (long long)(sq.q0 + tok) * a.out_stride + (long long)hd * D;
#pragma unroll
    for (int j = 0; j < (kParts + 3) / 4; ++j) {
        const int part = (threadIdx.x >> 6) + 4 * j;
        if (part < kParts)
            *(uint2*)(y + RW * (part / (VE / 4)) + Shape<RW>::at(part % (VE / 4) * 4, q)) = to16<BF16>(o[j] * inv);
    }
}

constexpr int kCus = 256;
constexpr int kLeast = 8;          // tiles of a piece

struct Launch {
    bool wide;                     // 256 rows a workgroup (128 at 256 columns), else 64
    int rows_each;
    long long units;               // at most
    int share;
    size_t ml, total;
};
static Launch plan_of(const xp_kv_dims* d, int heads, int rows, int batch, int max_len) {
    Launch p{};
    const long long pairs = (long long)rows * (heads / d->kv_heads);
    p.wide = d->head_dim == 256 || pairs >= 128ll * (batch < 1 ? 1 : batch);
    p.rows_each = !p.wide ? 64 : (d->head_dim == 256 ? 128 : 256);
    p.units = ((pairs + p.rows_each - 1) / p.rows_each + batch) * d->kv_heads;
    const int tiles = (int)(((long long)max_len + 63) / 64);
    const int per_cu = p.wide ? 1 : 2;
    p.share = tiles > kLeast ? kCus * per_cu : 0;
    p.ml = (size_t)2 * p.share * p.rows_each * d->head_dim * sizeof(float);
    p.total = p.ml + (size_t)2 * p.share * p.rows_each * 3 * sizeof(float);
    p.total = p.total ? p.total : 16;
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
static int launch(const Args& a, const Launch& p, hipStream_t s) {
    constexpr int RW = D == 256 ? 16 : 32;
    // what cutting adds is below one piece for each of `share` workgroups, for all kv heads of a piece
    const unsigned kv = (unsigned)a.g.kv_heads;
    const dim3 grid((unsigned)p.units + ((unsigned)p.share + kv - 1) / kv * kv);
    const unsigned cut = ((unsigned)p.share + kv - 1) / kv * kv;
    if (p.wide) {
        hipLaunchKernelGGL((attn_chunk_kernel<D, RW, 8, BF16>), grid, dim3(512), 0, s, a);
        if (p.share) hipLaunchKernelGGL((chunk_join_kernel<D, RW, 8, BF16>), dim3(8, cut), dim3(256), 0, s, a);
    } else if constexpr (D != 256) {
        hipLaunchKernelGGL((attn_chunk_kernel<D, 16, 4, BF16>), grid, dim3(256), 0, s, a);
        if (p.share) hipLaunchKernelGGL((chunk_join_kernel<D, 16, 4, BF16>), dim3(4, cut), dim3(256), 0, s, a);
    }
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
    if (ws_bytes < p.total) return XP_ERR_WORKSPACE;
    Args a{};
    a.g = kv::geo_of(dims, max_pages);
    a.q = (const uint16_t*)q;
    a.q_stride = q_stride;
    a.cache = cache;
    a.cu = cu_rows;
    a.start = start;
    a.table = table;
    a.out = (uint16_t*)out;
    a.out_stride = out_stride;
    a.part = (float*)workspace;
    a.part_ml = (float*)((char*)workspace + p.ml);
    a.batch = batch;
    a.rows = rows;
    a.group = heads / dims->kv_heads;
    a.window = window;
    a.share = p.share;
    a.least = kLeast;
    a.scale_m = (float)__builtin_frexp((double)scale * 1.4426950408889634, &a.scale_e);
    hipStream_t s = (hipStream_t)stream;
    const bool bf = type == XP_BF16;
    switch (dims->head_dim) {
        case 64: return bf ? launch<64, true>(a, p, s) : launch<64, false>(a, p, s);
        case 128: return bf ? launch<128, true>(a, p, s) : launch<128, false>(a, p, s);
        default: return bf ? launch<256, true>(a, p, s) : launch<256, false>(a, p, s);
    }
}
