// xp_attn_sparse.hip — attention of query rows over chosen blocks of the 4-bit cache:
// every (row, kv head) has its own list of 64-position blocks.
//
// A unit is a row, a kv head and up to 16 of its heads; its waves take the listed tiles in
// turn and join in LDS. What happens to a tile is what decode attention does (order of
// positions, precision: see xp_attn.hip). A lane looks up one entry of the list: which
// block, its page, and where its tile lies, 64 entries at once, so that no tile waits for a
// page number. Few units with long lists are cut into pieces, joined by a second launch.
//
// Bound by the tiles' bytes where they are read once, else by decoding them (vector pipes 66% busy
// where a kv head has 4 of the products' 16 columns): a step of 30 rows of 32 heads of 128, 8 kv heads,
// over 32 blocks each takes 19 us, 3.5 TB/s of tiles that are read once; 512 rows of a prompt over
// 16 blocks each share theirs and take 72 us, 7.9 TB/s out of the caches.
#include "xp_attn_dev.h"

namespace xp {
namespace sparse {

using namespace attn;
using kv::Geo;

struct Args {
    Geo g;
    const void* q;
    long long q_stride;
    const uint8_t* cache;
    const int32_t* cu;
    const int32_t* start;
    const int32_t* table;
    const int32_t* sel;
    void* out;
    long long out_stride;
    float* part;          // partial outputs of pieces, unscaled
    float* part_ml;       // their maxima, sums and the rows' factors
    int batch, group, head_blocks, keep;
    int pieces, each;     // of a list; entries of a piece
    float scale_m;        // scale * log2(e) = scale_m * 2^scale_e
    int scale_e;
};

template <int D>
constexpr int waves_per_cu() {
    return D == 64 ? 16 : (D == 128 ? 12 : 8);
}
template <int D, bool BF16>
__device__ __forceinline__ void store_out(const Args& a, int row, int head, int hb, int h, int c, int q, f32x4 o, float sum) {
    if (hb * 16 + c >= a.group) return;
    uint16_t* y = (uint16_t*)a.out + (long long)row * a.out_stride + (long long)(head * a.group + hb * 16 + c) * D;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;     // nothing seen: zeros
    *(uint2*)(y + 16 * h + 4 * q) = to16<BF16>(o * inv);
}

// ONE: a wave for each unit, which joins nothing; four of those fit a SIMD up to 128 columns.
template <int D, bool BF16, bool ONE>
__global__ __launch_bounds__((ONE ? 64 : 64 * waves_per_cu<D>()), (!ONE ? 1 : D == 64 ? 4 : D == 128 ? 3 : 2)) void attn_sparse_kernel(Args a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const int wave = ONE ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = ONE ? 1 : blockDim.x >> 6;
    // kv heads next to each other, so that the XCDs share out the heads of a row
    const int unit = blockIdx.x / a.pieces, piece = blockIdx.x - unit * a.pieces;
    const int head = unit % a.g.kv_heads, rest = unit / a.g.kv_heads, hb = rest % a.head_blocks, row = rest / a.head_blocks;
    const int b = kv::sequence_of_row(a.cu, a.batch, row);
    if (b >= a.batch) return;                  // rows behind the last sequence
    const int cap = a.g.max_pages * a.g.page, tiles = a.g.page >> 6;
    long long pos = (long long)a.start[b] + (row - a.cu[b]);
    const int at = pos < 0 ? -1 : (pos >= cap ? cap - 1 : (int)pos);
    const int32_t* tr = a.table + (long long)b * a.g.max_pages;
    const int32_t* list = a.sel + ((long long)row * a.g.kv_heads + head) * a.keep;
    const int end = (piece + 1) * a.each < a.keep ? (piece + 1) * a.each : a.keep;

    const int h0 = hb * 16 + c;                // the lane's head of the group
    h16x8 qf[Dim<D>::NW];
    const float factor = row_frags<D, BF16>((const uint16_t*)a.q + (long long)row * a.q_stride + (long long)(head * a.group + h0) * D,
                                            h0 < a.group, q, a.scale_m, a.scale_e, qf);
    Running<D> r;
    r.clear();
    uint8_t* region = lds + wave * wave_v_bytes<D>();
    walk_tiles<D>(
        a.cache, piece * a.each + wave, end, waves,
        [&](int i, long long& place) {
            const int blk = list[i];
            if (blk < 0 || blk > at >> 6) return -1;       // at is below the table's end
            const int col = blk / tiles, id = tr[col];
            place = (((long long)id * a.g.kv_heads + head) * tiles + (blk - col * tiles)) * kv::tile_bytes(Dim<D>::NG);
            return (unsigned)id < (unsigned)a.g.n_pages ? blk : -1;
        },
        [&](int base, f32x4 (&s)[4], VTile<D>& v) {
            if (base + 63 > at) {              // the row's own block: what lies behind it is not seen
#pragma unroll
                for (int bl = 0; bl < 4; ++bl)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (base + 16 * bl + 4 * q + e > at) s[bl][e] = -__builtin_inff();
                clear_v<D>(v, at + 1 - base, lane);
            }
            return false;                      // all heads see the same
        },
        [](int) {}, qf, factor, r, region);
    if constexpr (ONE) {
        r.l = sum_over_q(r.l);
#pragma unroll
        for (int h = 0; h < Dim<D>::NH; ++h) store_out<D, BF16>(a, row, head, hb, h, c, q, r.o[h], r.l);
        return;
    }
    join_waves<D>(r, factor, lds, wave, waves, [&](int h, f32x4 o, float m, float l) {
        if (a.pieces == 1) {
            store_out<D, BF16>(a, row, head, hb, h, c, q, o, l);
            return;
        }
        const long long slot = blockIdx.x;
        ((f32x4*)a.part)[(slot * Dim<D>::NH + h) * 64 + lane] = o;
        if (h == 0 && q == 0) {
            float* pm = a.part_ml + slot * 48 + c;
            pm[0] = m;
            pm[16] = l;
            pm[32] = factor;
        }
    });
}

// Joins a unit's pieces, in order: a wave takes four columns of 16 heads a lane.
template <int D, bool BF16>
__global__ __launch_bounds__(64) void sparse_join_kernel(Args a) {
    constexpr int NH = Dim<D>::NH;
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const int h = blockIdx.x % NH, unit = blockIdx.x / NH;
    const int head = unit % a.g.kv_heads, rest = unit / a.g.kv_heads, hb = rest % a.head_blocks, row = rest / a.head_blocks;
    if (kv::sequence_of_row(a.cu, a.batch, row) >= a.batch) return;
    const long long slot = (long long)unit * a.pieces;
    const f32x4* po = (const f32x4*)a.part + (slot * NH + h) * 64 + lane;
    const float* pm = a.part_ml + slot * 48 + c;
    const float fr = pm[32];
    float m = -__builtin_inff(), l = 0.0f;
    f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.pieces; ++s) m = fmaxf(m, pm[s * 48]);
    const float safe = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll 4
    for (int s = 0; s < a.pieces; ++s) {
        const float f = __builtin_amdgcn_exp2f((pm[s * 48] - safe) * fr);
        l = __builtin_fmaf(pm[s * 48 + 16], f, l);
        o += po[(long long)s * (NH * 64)] * f;
    }
    store_out<D, BF16>(a, row, head, hb, h, c, q, o, l);
}

constexpr int kCus = 256;
// Units from which a wave takes one whole, without a join. Lists of 16 blocks, 128 columns, a wave and
// four waves a unit: 1,024 units 30 and 27 us, 2,048 42 and 44, 4,096 72 and 82, 8,192 127 and 149; eight
// waves a unit take 131 us at 4,096. At 2,048 units 64 columns 27 and 27, 256 columns 38 and 51.
constexpr int kOneWave = 8 * kCus;

struct Launch {
    long long units;
    int head_blocks, waves, pieces, each;
    size_t part, total;
};
static Launch plan_of(const xp_kv_dims* d, int heads, int rows, int keep) {
    Launch p{};
    p.head_blocks = (heads / d->kv_heads + 15) / 16;
    p.units = (long long)rows * d->kv_heads * p.head_blocks;
    const int most = d->head_dim == 64 ? waves_per_cu<64>() : d->head_dim == 128 ? waves_per_cu<128>() : waves_per_cu<256>();
    // Units enough for all waves are one's each; enough for two a CU, four waves'; fewer take all the
    // waves that a CU has, and where their lists are long, several CUs.
    p.pieces = 1;
    if (p.units >= kOneWave) {
        p.waves = 1;
    } else if (p.units >= 2 * kCus) {
        p.waves = keep < 4 ? keep : 4;
    } else {
        p.waves = keep < most ? keep : most;
        const long long room = kCus / (p.units < 1 ? 1 : p.units), rounds = (keep + 2 * p.waves - 1) / (2 * p.waves);
        p.pieces = (int)(rounds < 2 || room < 2 ? 1 : (rounds < room ? rounds : room));
    }
    p.each = (keep + p.pieces - 1) / p.pieces;
    p.pieces = (keep + p.each - 1) / p.each;
    p.part = p.pieces > 1 ? (size_t)p.units * p.pieces * 16 * d->head_dim * sizeof(float) : 0;
    p.total = p.pieces > 1 ? p.part + (size_t)p.units * p.pieces * 48 * sizeof(float) : 16;
    return p;
}

static int check_sparse(const xp_kv_dims* d, int heads, int batch, int max_pages, int rows, int keep) {
    const int st = kv::check_geo(d, batch, max_pages);
    if (st != XP_OK) return st;
    if (heads < 1 || heads > 65535 || heads % d->kv_heads || rows < 0 || keep < 1 || keep > (1 << 24)) return XP_ERR_SHAPE;
    // four waves of each unit, or its join's blocks: a launch has fewer than 2^32 threads
    if ((long long)rows * d->kv_heads * ((heads / d->kv_heads + 15) / 16) >= (1 << 24)) return XP_ERR_SHAPE;
    return XP_OK;
}

template <int D, bool BF16>
static int launch(const Args& a, const Launch& p, hipStream_t s) {
    static_assert(wave_join_bytes<D>() >= wave_v_bytes<D>());
    const dim3 grid((unsigned)(p.units * p.pieces)), block(64 * p.waves);
    if (p.waves == 1 && p.pieces == 1)
        hipLaunchKernelGGL((attn_sparse_kernel<D, BF16, true>), grid, block, wave_v_bytes<D>(), s, a);
    else
        hipLaunchKernelGGL((attn_sparse_kernel<D, BF16, false>), grid, block, p.waves * wave_join_bytes<D>(), s, a);
    if (p.pieces > 1)
        hipLaunchKernelGGL((sparse_join_kernel<D, BF16>), dim3((unsigned)(p.units * Dim<D>::NH)), dim3(64), 0, s, a);
    return launch_status();
}

}  // namespace sparse
}  // namespace xp

using namespace xp;
using namespace xp::sparse;

XP_API size_t xp_attn_sparse_workspace_bytes(const xp_kv_dims* dims, int32_t heads, int32_t rows, int32_t keep) {
    if (check_sparse(dims, heads, 1, 1, rows, keep) != XP_OK) return 0;
    return plan_of(dims, heads, rows, keep).total;
}

XP_API int xp_attn_sparse(const xp_kv_dims* dims, int32_t heads, int32_t batch, int32_t max_pages, int32_t rows, int32_t keep,
                          int32_t type, const void* q, int64_t q_stride, float scale, const uint8_t* cache,
                          const int32_t* table, const int32_t* cu_rows, const int32_t* start, const int32_t* sel, void* out,
                          int64_t out_stride, void* workspace, size_t ws_bytes, void* stream) {
    const int st = check_sparse(dims, heads, batch, max_pages, rows, keep);
    if (st != XP_OK) return st;
    if ((type != XP_BF16 && type != XP_F16) || !(scale > 0.0f && scale < __builtin_inff())) return XP_ERR_SHAPE;
    if (batch == 0 || rows == 0) return XP_OK;
    if (!q || !cache || !table || !cu_rows || !start || !sel || !out || !workspace) return XP_ERR_NULL;
    const int64_t width = (int64_t)heads * dims->head_dim;
    if (q_stride < width || out_stride < width || q_stride % 8 || out_stride % 4 || !kv::aligned_to(q, 16) ||
        !kv::aligned_to(out, 8) || !kv::aligned_to(cache, 16) || !kv::aligned_to(table, 4) || !kv::aligned_to(cu_rows, 4) ||
        !kv::aligned_to(start, 4) || !kv::aligned_to(sel, 4) || !kv::aligned_to(workspace, 16))
        return XP_ERR_SHAPE;
    const Launch p = plan_of(dims, heads, rows, keep);
    // a unit's q is read before its heads are written, but every piece reads it
    const kv::Rows qr{q, rows, 2 * q_stride, 2 * width}, yr{out, rows, 2 * out_stride, 2 * width};
    if (!qr.same(yr) && kv::rows_meet(qr, yr)) return XP_ERR_SHAPE;
    // what other units still read
    const kv::Rows read[] = {kv::flat(sel, (int64_t)rows * dims->kv_heads * keep * 4), kv::flat(cache, (int64_t)xp_kv_bytes(dims)),
                             kv::flat(table, 4 * (int64_t)batch * max_pages), kv::flat(cu_rows, 4 * (int64_t)batch + 4),
                             kv::flat(start, 4 * (int64_t)batch), qr, yr};
    if (kv::meets_any(yr, read, 5)) return XP_ERR_SHAPE;
    if (p.pieces > 1 && kv::meets_any(kv::flat(workspace, (int64_t)(ws_bytes < p.total ? ws_bytes : p.total)), read, 7)) return XP_ERR_SHAPE;
    if (ws_bytes < p.total) return XP_ERR_WORKSPACE;
    Args a{};
    a.g = kv::geo_of(dims, max_pages);
    a.q = q;
    a.q_stride = q_stride;
    a.cache = cache;
    a.cu = cu_rows;
    a.start = start;
    a.table = table;
    a.sel = sel;
    a.out = out;
    a.out_stride = out_stride;
    a.part = (float*)workspace;
    a.part_ml = (float*)((char*)workspace + p.part);
    a.batch = batch;
    a.group = heads / dims->kv_heads;
    a.head_blocks = p.head_blocks;
    a.keep = keep;
    a.pieces = p.pieces;
    a.each = p.each;
    a.scale_m = (float)__builtin_frexp((double)scale * 1.4426950408889634, &a.scale_e);
    hipStream_t s = (hipStream_t)stream;
    const bool bf = type == XP_BF16;
    switch (dims->head_dim) {
        case 64: return bf ? launch<64, true>(a, p, s) : launch<64, false>(a, p, s);
        case 128: return bf ? launch<128, true>(a, p, s) : launch<128, false>(a, p, s);
        default: return bf ? launch<256, true>(a, p, s) : launch<256, false>(a, p, s);
    }
}
