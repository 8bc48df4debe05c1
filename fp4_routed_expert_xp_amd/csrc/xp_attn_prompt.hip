// xp_attn_prompt.hip — causal attention over whole prompts, packed sequences of
// different lengths, grouped heads, bf16 or fp16.
//
// One pass over the keys with a running maximum and sum. A row is a (token, head of
// the kv head's group) pair, tokens first, so the heads that share keys share a
// workgroup and a short prompt still fills its rows. A wave owns RW rows and takes
// 64 positions at a time. S^T = K Q^T (v_mfma_f32_32x32x16 for 32 rows, 16x16x32 for
// 16; positions as the matrix rows) leaves lane (m, q) = (lane % RW, lane / RW) with
// row m at every fourth quad of positions, so the exponentials, once rounded, are the
// operand of O^T += V^T P^T where they are: V follows the same order of positions
// through the 16-bit transposing LDS read, which hands a lane four positions of one
// column.
//
// Waves of 32 rows read k and v from LDS half as often; their registers (outputs,
// scores, q) leave two waves a SIMD up to 128 columns and one at 256, where waves of 16
// rows leave two: 8 heads of 256 over 4,096 rows take 158 us in those and took 233 in
// waves of 32, 32 heads of 128 over 8,192 rows 797 us in waves of 16 and 586 in 32
// (938 TFLOP/s of the pairs that are seen; a large bf16 product runs at 1,380 here).
// Bound there by both pipes in turn: of the SIMDs' time the matrix pipe is busy 42%,
// the vector pipe 39% (the exponentials two fifths of it), both at once 11%. Much of the
// rest is waiting for the tile ahead: it is asked for at the top of a tile, but the wait
// that the compiler puts before the tile's first read of K, whose loads to LDS it cannot
// tell from the ones just begun, is for all loads in flight. LDS itself is busy 21%,
// without bank conflicts.
//
// Scores, maxima, sums and outputs are fp32; exponentials round once to the type of
// v (the product's operand; in fp16 as 2^13 times the weight, so that a long tail of
// small weights is not lost), the result once to the output type.
#include "xp_kv_dev.h"

namespace xp {
namespace prompt {

typedef __attribute__((ext_vector_type(8))) _Float16 h16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 b16x8;
typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) short s16x2;

typedef __attribute__((address_space(3))) void* lptr;
typedef __attribute__((address_space(1))) const void* gptr;

constexpr int kPos = 64;     // positions of a tile
// Up to this many workgroups of 128 rows (two for each CU) they are of 64 rows, in waves
// of 16: each CU's chain of tiles is shorter. 2,000 rows of 16/8 heads of 128 (264
// workgroups) take 48 us so and 57 us in 128 rows, 1,000 of 32/8 28 and 33; 2,000 of
// 32/8 (512) 57 and 60; eight packed prompts to 1,000 (1,190) 80 and 61.
constexpr int kFew = 512;
// In powers of two: by how much the running maximum may lag behind, and what exponentials are
// held as times the weight. fp16 has the range for both only together (15), so it lags less:
// weights down to 2^-27 of the largest then keep all their bits, and what is below is within
// 2^-38 of it. bf16 has fp32's range.
constexpr float lag_of(bool bf16) { return bf16 ? 8.0f : 2.0f; }
constexpr float lift_of(bool bf16) { return bf16 ? 0.0f : 13.0f; }
constexpr float kNear = 256.0f;   // maxima in log2 units up to which a product with the factor is used

struct Args {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* out;
    long long q_stride, k_stride, v_stride, out_stride;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int rows_q, rows_k, batch, kv_heads, group, window;
    float scale_log2;
    float lag;            // lag_of in units of the scores
};

// What a wave of RW rows has of its products: RW x RW results, VE a lane, over KD of
// the contraction; lane (m, q) holds column m and, as element r, row at(r, q).
template <int RW>
struct Shape {
    static constexpr int VE = RW * RW / 64, KD = 512 / RW, NQ = 64 / RW;
    typedef __attribute__((ext_vector_type(VE))) float acc;
    static __device__ __forceinline__ int at(int r, int q) { return 4 * NQ * (r >> 2) + 4 * q + (r & 3); }
};
template <int RW, bool BF16>
__device__ __forceinline__ typename Shape<RW>::acc mma(s16x8 a, s16x8 b, typename Shape<RW>::acc c) {
    if constexpr (RW == 32 && BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b16x8, a), __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
    else if constexpr (RW == 32)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h16x8, a), __builtin_bit_cast(h16x8, b), c, 0, 0, 0);
    else if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, a), __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8, a), __builtin_bit_cast(h16x8, b), c, 0, 0, 0);
}

// 16 bits of the operand type, nearest even.
template <bool BF16>
__device__ __forceinline__ short half_of(float x) {
    if constexpr (BF16) return __builtin_bit_cast(short, (__bf16)x);
    return __builtin_bit_cast(short, (_Float16)x);
}

// c + the two halves of a pair.
template <bool BF16>
__device__ __forceinline__ float plus_pair(s16x2 a, float c) {
    if constexpr (BF16) {
        typedef __attribute__((ext_vector_type(2))) __bf16 b16x2;
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b16x2, a), b16x2{(__bf16)1.0f, (__bf16)1.0f}, c, false);
    } else {
        typedef __attribute__((ext_vector_type(2))) _Float16 h16x2;
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(h16x2, a), h16x2{(_Float16)1.0f, (_Float16)1.0f}, c, false);
    }
}

template <bool BF16>
__device__ __forceinline__ bool not_finite(uint16_t u) {
    constexpr uint16_t e = BF16 ? 0x7f80 : 0x7c00;
    return (u & e) == e;
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

// LDS places. K: a row's 16-byte chunks are permuted so that 16 neighbouring rows at
// one chunk index cover all banks; V: its blocks of RW columns, so that the rows of a
// transposing read (eight of 64 bytes, or sixteen of 32) meet each bank twice at most.
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
// Chunk of 16 bytes of a row of v that LDS chunk c of the row holds.
template <int D, int RW>
__device__ __forceinline__ int v_chunk(int pos, int c) {
    constexpr int per = RW / 8;                // chunks of a block
    return (v_at<D, RW>(pos, c / per) - pos * (2 * D)) / 16 + c % per;
}

__device__ __forceinline__ s16x8 v_frag(const uint8_t* a, const uint8_t* b) {
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)a);
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)b);
    return s16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
}

// A tile that some row does not see whole and that holds values of v that are not
// finite: a zero weight times one of those is NaN, so they are taken out of the tile
// and added here, to the rows that see them. One product per kind (+inf, -inf, NaN)
// of its places with what each row sees counts the seen ones of each column.
template <int D, int RW, bool BF16>
__device__ __forceinline__ void set_apart(typename Shape<RW>::acc (&o)[D / RW], const uint8_t* lv, int first, int at, int lo) {
    constexpr short one = BF16 ? 0x3f80 : 0x3c00;
    constexpr uint16_t inf = BF16 ? 0x7f80 : 0x7c00;
    constexpr int KD = Shape<RW>::KD, VE = Shape<RW>::VE;
    const int lane = threadIdx.x & 63, q = lane / RW;
    const int row = 4 * q + ((lane & 15) >> 2), col = ((lane % RW) >> 4) * 32 + (lane & 3) * 8;
#pragma unroll
    for (int d = 0; d < D / RW; ++d)
#pragma unroll 1
        for (int kind = 0; kind < 3; ++kind) {
            typename Shape<RW>::acc n;
#pragma unroll
            for (int r = 0; r < VE; ++r) n[r] = 0.0f;
#pragma unroll 1
            for (int st = 0; st < kPos / KD; ++st) {
                const int pos = KD * st + row;
                const s16x8 vf = v_frag(lv + v_at<D, RW>(pos, d) + col, lv + v_at<D, RW>(pos + KD / 2, d) + col);
                s16x8 f, seen;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint16_t u = (uint16_t)vf[j];
                    const bool is = kind == 0 ? u == inf : (kind == 1 ? u == (inf | 0x8000)
                                                                      : not_finite<BF16>(u) && (u & 0x7fff) != inf);
                    f[j] = is ? one : (short)0;
                    const int ps = first + KD * st + KD / 2 * (j >> 2) + 4 * q + (j & 3);
                    seen[j] = ps <= at && ps >= lo ? one : (short)0;
                }
                n = mma<RW, BF16>(f, seen, n);
            }
            const float add = kind == 0 ? __builtin_inff() : (kind == 1 ? -__builtin_inff() : __builtin_nanf(""));
#pragma unroll
            for (int r = 0; r < VE; ++r)
                if (n[r] > 0.0f) o[d][r] += add;
        }
}

template <int ROWS>
__device__ __forceinline__ int blocks_of(const Args& a, int b) {
    if (b >= a.batch) return 0;
    const long long rows = (long long)a.cu_q[b + 1] - a.cu_q[b];
    return rows > 0 && rows <= a.rows_q ? (int)((rows * a.group + ROWS - 1) / ROWS) : 0;
}
// The workgroup's block of rows: sequence and first row. The blocks that run longest,
// the last ones of their sequences, come first, so that short ones fill the gaps at the
// end: among up to 64 sequences by their number in the sequence, else each sequence's
// from its last to its first. false: no such block.
template <int ROWS>
__device__ __forceinline__ bool find_block(const Args& a, int blk, int& seq, int& first) {
    const int lane = threadIdx.x & 63;
    if (a.batch <= 64) {
        const int n = blocks_of<ROWS>(a, lane);
        // blocks numbered k or more: the sum of max(0, n - k); find the k of block blk
        const auto from = [&](int k) { return __builtin_amdgcn_readlane(wave_incl_sum(n > k ? n - k : 0), 63); };
        if (blk >= from(0)) return false;
        int lo = 0, hi = (int)wave_max_u32((uint32_t)n);       // from(lo) > blk >= from(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (from(mid) > blk)
                lo = mid;
            else
                hi = mid;
        }
        const uint64_t there = __ballot(n > lo);
        const int at = blk - from(lo + 1);
        const uint64_t hit = __ballot(n > lo && __popcll(there & ((1ull << lane) - 1)) == at);
        seq = __ffsll((unsigned long long)hit) - 1;
        first = lo * ROWS;
        return true;
    }
    int total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int before = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 64) {
            const int n = blocks_of<ROWS>(a, b0 + lane);
            const int incl = wave_incl_sum(n);
            if (pass == 1) {
                const uint64_t hit = __ballot(n > 0 && before + incl - n <= blk && blk < before + incl);
                if (hit) {
                    const int l = __ffsll((unsigned long long)hit) - 1;
                    seq = b0 + l;
                    first = (blk - before - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(n, l))) * ROWS;
                    return true;
                }
            }
            before += __builtin_amdgcn_readlane(incl, 63);
        }
        if (pass == 0) {
            total = before;
            if (blk >= total) return false;
            blk = total - 1 - blk;
        }
    }
    return false;
}

template <int D, int RW, int ROWS, bool BF16>
__global__ __launch_bounds__(64 * ROWS / RW, 2) void attn_prompt_kernel(Args a) {
    typedef Shape<RW> Sh;
    typedef typename Sh::acc acc;
    constexpr int KD = Sh::KD, VE = Sh::VE, kThreads = 64 * ROWS / RW;
    constexpr int NS = D / KD;                 // contraction steps of the scores
    constexpr int NT = kPos / RW;              // blocks of positions of the scores
    constexpr int ND = D / RW;                 // column blocks of the output
    constexpr int NL = kPos * D / 8 / kThreads;   // 16-byte chunks a thread stages of each of k and v
    constexpr int kTile = kPos * D * 2;        // bytes of a tile of k, or of v
    constexpr float kLift = lift_of(BF16);
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][2 * kTile];

    const int tid = threadIdx.x, lane = tid & 63, m = lane % RW, q = lane / RW;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int head = blockIdx.x % a.kv_heads;
    int b, first;
    if (!find_block<ROWS>(a, blockIdx.x / a.kv_heads, b, first)) return;
    const int q0 = a.cu_q[b], nq = a.cu_q[b + 1] - q0;
    if (q0 < 0 || (long long)q0 + nq > a.rows_q) return;
    int k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    k0 = k0 < 0 ? 0 : (k0 > a.rows_k ? a.rows_k : k0);
    k1 = k1 < k0 ? k0 : (k1 > a.rows_k ? a.rows_k : k1);
    const int nk = k1 - k0, shift = nk - nq;   // token i sits at position i + shift

    const int rows = nq * a.group;
    const int row = first + wave * RW + m;
    const bool live = row < rows;
    const int tok = live ? row / a.group : 0;
    const int hd = head * a.group + (live ? row - tok * a.group : 0);
    const int at = live ? tok + shift : -1;    // the row's own position
    const int lo = kv::first_seen(at, a.window);

    s16x8 qf[NS];
    const uint16_t* qp = a.q + (long long)(q0 + tok) * a.q_stride + (long long)hd * D + 8 * q;
#pragma unroll
    for (int st = 0; st < NS; ++st) qf[st] = live ? *(const s16x8*)(qp + KD * st) : s16x8{0, 0, 0, 0, 0, 0, 0, 0};

    // tiles that some row of the workgroup sees, and those that all see whole
    const int last_row = first + ROWS < rows ? first + ROWS - 1 : rows - 1;
    const int at_first = first / a.group + shift, at_last = last_row / a.group + shift;
    const int t_hi = at_last >= 0 ? (at_last >> 6) + 1 : 0;
    const int t_lo = kv::first_seen(at_first, a.window) >> 6;
    const int full_lo = kv::first_seen(at_last, a.window), full_hi = at_first + 1;

    acc o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < VE; ++r) o[d][r] = 0.0f;
    float mx = -__builtin_inff(), sum = 0.0f;
    uint64_t far = 0;                          // lanes whose maximum is too large for that

    const uint16_t* kp = a.k + (long long)k0 * a.k_stride + (long long)head * D;
    const uint16_t* vp = a.v + (long long)k0 * a.v_stride + (long long)head * D;
    // A tile goes straight from memory to LDS, asked for one tile ahead, into the other buffer: the
    // j-th load of a thread fills LDS chunk j * kThreads + tid, and reads the chunk that the
    // permutation above puts there. Rows behind the last key repeat it (no row sees them).
    const int lp = tid / (D / 8), lc = tid % (D / 8);
    constexpr int kStep = kThreads / (D / 8);  // positions that one load of all threads covers: whole
    static_assert(kStep % 16 == 0);            // sixteens, which the permutations repeat after
    const int kc = (k_at<D>(lp, lc) - lp * (2 * D)) / 16, vc = v_chunk<D, RW>(lp, lc);
    const uint32_t k_off = 2 * ((uint32_t)lp * (uint32_t)a.k_stride + 8 * kc);   // bytes from a load's first position
    const uint32_t v_off = 2 * ((uint32_t)lp * (uint32_t)a.v_stride + 8 * vc);
    auto fetch = [&](int tile, uint8_t* to) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int p = tile * kPos + j * kStep, over = p + lp - (nk - 1);
            const uint8_t* kj = (const uint8_t*)(kp + (long long)p * a.k_stride);
            const uint8_t* vj = (const uint8_t*)(vp + (long long)p * a.v_stride);
            uint8_t* d = to + j * (16 * kThreads) + wave * 1024;
            if (tile * kPos + kPos <= nk) {
                __builtin_amdgcn_global_load_lds((gptr)(kj + k_off), (lptr)d, 16, 0, 0);
                __builtin_amdgcn_global_load_lds((gptr)(vj + v_off), (lptr)(d + kTile), 16, 0, 0);
            } else {
                const long long back = over > 0 ? over : 0;
                __builtin_amdgcn_global_load_lds((gptr)(kj + k_off - 2 * back * a.k_stride), (lptr)d, 16, 0, 0);
                __builtin_amdgcn_global_load_lds((gptr)(vj + v_off - 2 * back * a.v_stride), (lptr)(d + kTile), 16, 0, 0);
            }
        }
    };
    if (t_lo < t_hi) fetch(t_lo, lds[0]);

    for (int tile = t_lo; tile < t_hi; ++tile) {
        const bool masked = tile * kPos < full_lo || tile * kPos + kPos > full_hi;
        uint8_t* lk = lds[(tile - t_lo) & 1];
        uint8_t* lv = lk + kTile;
        // this wave's loads of the tile have landed, its reads of the last one are done; then everyone's
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (tile + 1 < t_hi) fetch(tile + 1, lds[(tile + 1 - t_lo) & 1]);
        bool bad = false;
        if (masked) {
            uint32_t carry = 0;
            // a value of v that is not finite must not meet the zero weight of a row that does not see it
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const uint4 c = *(const uint4*)(lv + (j * kThreads + tid) * 16);
                // all exponent bits set: adding the lowest of them carries into the sign's place
                constexpr uint32_t e = BF16 ? 0x7f807f80u : 0x7c007c00u, low = BF16 ? 0x00800080u : 0x04000400u;
                carry |= ((c.x & e) + low) | ((c.y & e) + low) | ((c.z & e) + low) | ((c.w & e) + low);
            }
            bad = __syncthreads_or((carry & 0x80008000u) != 0);
        }

        acc s[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < VE; ++r) s[t][r] = 0.0f;
#pragma unroll
        for (int st = 0; st < NS; ++st)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                s[t] = mma<RW, BF16>(*(const s16x8*)(lk + k_at<D>(RW * t + m, KD / 8 * st + q)), qf[st], s[t]);
        if (masked) {
            const int here = tile * kPos + 4 * q;
#pragma unroll
            for (int e = 0; e < NT * VE; ++e)
                if (RW * (e / VE) + Sh::at(e % VE, 0) > at - here) s[e / VE][e % VE] = -__builtin_inff();
            if (a.window > 0)
#pragma unroll
                for (int e = 0; e < NT * VE; ++e)
                    if (RW * (e / VE) + Sh::at(e % VE, 0) < lo - here) s[e / VE][e % VE] = -__builtin_inff();
        }
        float top = s[0][0];
#pragma unroll
        for (int e = 1; e < NT * VE; ++e) top = fmaxf(top, s[e / VE][e % VE]);
        top = over_q<RW, false>(top);
        // Exponentials are taken from a maximum that lags behind, so what was summed needs no
        // factor but in a row's first tiles. mx is the score as it is. Up to kNear in log2 units
        // its product with the factor, rounded, is within 2^-16 of the maximum, far below the
        // exponentials' own rounding, and one fma does; beyond that the factor multiplies
        // differences only, which is right at any size, and nothing lags.
        if (__builtin_expect((__ballot(top > mx + a.lag) | far) != 0, 0)) {
            const float nm = fmaxf(top, mx), from = nm == -__builtin_inff() ? 0.0f : nm;
            const float alpha = __builtin_amdgcn_exp2f((mx - from) * a.scale_log2);
            mx = nm;
            far = __ballot(!(__builtin_fabsf(from * a.scale_log2) <= kNear));
            if (far)
#pragma unroll
                for (int e = 0; e < NT * VE; ++e) s[e / VE][e % VE] -= from;
            sum *= alpha;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] *= alpha;
        }
        const float base = far || mx == -__builtin_inff() ? kLift : __builtin_fmaf(-mx, a.scale_log2, kLift);
        // The sum is of the rounded exponentials, two at a time: what rounding adds to a weight
        // that stands out it adds to the sum as well (a maximum that lags is not 1 exactly).
        s16x8 p[NT * VE / 8];
#pragma unroll
        for (int e = 0; e < NT * VE; e += 2) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e / VE][e % VE], a.scale_log2, base));
            const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[(e + 1) / VE][(e + 1) % VE], a.scale_log2, base));
            const s16x2 xy = s16x2{half_of<BF16>(x), half_of<BF16>(y)};
            p[e >> 3][e & 7] = xy.x;
            p[e >> 3][(e & 7) + 1] = xy.y;
            sum = plus_pair<BF16>(xy, sum);
        }

        if (masked && bad) {
            set_apart<D, RW, BF16>(o, lv, tile * kPos, at, lo);
            __syncthreads();                   // every wave has seen the tile as it was
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                uint16_t* e = (uint16_t*)(lv + (j * kThreads + tid) * 16);
                for (int i = 0; i < 8; ++i)
                    if (not_finite<BF16>(e[i])) e[i] = 0;
            }
            __syncthreads();
        }
        const int vrow = 4 * q + ((lane & 15) >> 2), col = (m >> 4) * 32 + (lane & 3) * 8;
#pragma unroll
        for (int st = 0; st < kPos / KD; ++st)
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const int pos = KD * st + vrow;
                o[d] = mma<RW, BF16>(v_frag(lv + v_at<D, RW>(pos, d) + col, lv + v_at<D, RW>(pos + KD / 2, d) + col), p[st], o[d]);
            }
    }

    sum = over_q<RW, true>(sum);
    if (!live) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;      // nothing seen: zeros
    uint16_t* y = a.out + (long long)(q0 + tok) * a.out_stride + (long long)hd * D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
            uint32_t w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                w[j] = (uint32_t)(uint16_t)half_of<BF16>(o[d][e + 2 * j] * inv) |
                       (uint32_t)(uint16_t)half_of<BF16>(o[d][e + 2 * j + 1] * inv) << 16;
            *(uint2*)(y + RW * d + Sh::at(e, q)) = uint2{w[0], w[1]};
        }
}

}  // namespace prompt
}  // namespace xp

using namespace xp;
using namespace xp::prompt;

XP_API int xp_attn_prompt(int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t batch, int32_t rows_q, int32_t rows_k,
                          int32_t type, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, float scale, int32_t window,
                          void* out, int64_t out_stride, void* stream) {
    if (kv_heads < 1 || kv_heads > 1024 || heads < 1 || heads > 65535 || heads % kv_heads ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256) || batch < 0 || batch > 65535 || rows_q < 0 || rows_k < 0 ||
        (type != XP_BF16 && type != XP_F16) || window < 0 || !(scale > 0.0f && scale < __builtin_inff()))
        return XP_ERR_SHAPE;
    const int group = heads / kv_heads;
    // workgroups of 64 rows, the smaller of the two kinds
    const int64_t small = ((int64_t)rows_q * group + 63) / 64 + batch, large = ((int64_t)rows_q * group + 127) / 128 + batch;
    if ((int64_t)rows_q * group > 0x7fffffff - 128 || rows_k > 0x7fffffff - kPos || small * kv_heads >= (1 << 23))   // a launch has fewer than 2^32 threads
        return XP_ERR_SHAPE;
    if (batch == 0 || rows_q == 0) return XP_OK;
    if (!q || !cu_q || !cu_k || !out || (rows_k > 0 && (!k || !v))) return XP_ERR_NULL;
    const int64_t qw = (int64_t)heads * head_dim, kw = (int64_t)kv_heads * head_dim;
    const int64_t far = (int64_t)1 << 24;   // a load's offsets within 32 rows of k and v are 32-bit
    if (k_stride >= far || v_stride >= far) return XP_ERR_SHAPE;
    if (q_stride < qw || out_stride < qw || k_stride < kw || v_stride < kw || q_stride % 8 || k_stride % 8 || v_stride % 8 ||
        out_stride % 4 || !kv::aligned_to(q, 16) || !kv::aligned_to(k, 16) || !kv::aligned_to(v, 16) || !kv::aligned_to(out, 8) || !kv::aligned_to(cu_q, 4) || !kv::aligned_to(cu_k, 4))
        return XP_ERR_SHAPE;
    // a workgroup's q is read before its rows are written; k and v are read by all
    const kv::Rows qr{q, rows_q, 2 * q_stride, 2 * qw}, yr{out, rows_q, 2 * out_stride, 2 * qw};
    if ((!qr.same(yr) && kv::rows_meet(qr, yr)) || kv::rows_meet(kv::Rows{k, rows_k, 2 * k_stride, 2 * kw}, yr) ||
        kv::rows_meet(kv::Rows{v, rows_k, 2 * v_stride, 2 * kw}, yr))
        return XP_ERR_SHAPE;
    const float f = kv::log2_scale(scale);
    const float lag = lag_of(type == XP_BF16) / f;
    const Args a{(const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v, (uint16_t*)out, q_stride, k_stride, v_stride,
                 out_stride, cu_q, cu_k, rows_q, rows_k, batch, kv_heads, group, window, f,
                 lag < 0x1p127f ? lag : 0x1p127f};   // finite: the maximum may be -infinity
    hipStream_t s = (hipStream_t)stream;
#define XP_PROMPT_LAUNCH(D_, RW_, ROWS_, BLOCKS_)                                                  \
    do {                                                                                           \
        const dim3 grid((unsigned)(BLOCKS_ * kv_heads)), block(64 * ROWS_ / RW_);                  \
        if (type == XP_BF16)                                                                       \
            hipLaunchKernelGGL((attn_prompt_kernel<D_, RW_, ROWS_, true>), grid, block, 0, s, a);  \
        else                                                                                       \
            hipLaunchKernelGGL((attn_prompt_kernel<D_, RW_, ROWS_, false>), grid, block, 0, s, a); \
    } while (0)
    const bool few = large * kv_heads <= kFew;
    if (head_dim == 256)
        XP_PROMPT_LAUNCH(256, 16, 128, large);
    else if (head_dim == 128 && few)
        XP_PROMPT_LAUNCH(128, 16, 64, small);
    else if (head_dim == 128)
        XP_PROMPT_LAUNCH(128, 32, 128, large);
    else if (few)
        XP_PROMPT_LAUNCH(64, 16, 64, small);
    else
        XP_PROMPT_LAUNCH(64, 32, 128, large);
#undef XP_PROMPT_LAUNCH
    return launch_status();
}
