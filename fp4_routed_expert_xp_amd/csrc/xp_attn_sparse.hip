// xp_attn_sparse.hip — attention of query rows over chosen blocks of the 4-bit cache:
// every (row, kv head) has its own list of 64-position blocks.
//
// A unit is a row, a kv head and up to 16 of its heads; its waves take the listed tiles in
// turn and join in LDS. What happens to a tile is what decode attention does (order of
// positions, precision: see xp_attn.hip). A lane looks up one entry of the list: which
// block, its page, and where its tile lies, 64 entries at once, so that no tile waits for a
// page number. Few units with long lists are cut into pieces, joined by a second launch.
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

// q of 16 heads as fp16 fragments and their score factors; a head that is not there is 0.
template <int D, bool BF16>
__device__ __forceinline__ float load_q(const Args& a, int row, int head, int hb, int c, int q, h16x8 (&qf)[Dim<D>::NW]) {
    const int h = hb * 16 + c;
    const uint16_t* p = (const uint16_t*)a.q + (long long)row * a.q_stride + (long long)(head * a.group + (h < a.group ? h : 0)) * D;
    uint4 v[Dim<D>::NW];
#pragma unroll
    for (int w = 0; w < Dim<D>::NW; ++w) v[w] = h < a.group ? *(const uint4*)(p + dims_of<D>(q, w)) : uint4{0, 0, 0, 0};
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
    return fminf(fmaxf(__builtin_amdgcn_ldexpf(a.scale_m, a.scale_e - k), 0x1p-126f), 0x1p127f);
}

template <int D>
constexpr int waves_per_cu() {
    return D == 64 ? 16 : (D == 128 ? 12 : 8);
}
template <int D>
constexpr int region_bytes() {
    return Dim<D>::kVBytes + Dim<D>::NG * 64;
}
template <int D>
constexpr int join_bytes() {
    return Dim<D>::NH * 1024 + 128;
}

template <int D, bool BF16>
__device__ __forceinline__ void store_out(const Args& a, int row, int head, int hb, int h, int c, int q, f32x4 o, float sum) {
    if (hb * 16 + c >= a.group) return;
    uint16_t* y = (uint16_t*)a.out + (long long)row * a.out_stride + (long long)(head * a.group + hb * 16 + c) * D;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;     // nothing seen: zeros
    *(uint2*)(y + 16 * h + 4 * q) = to16<BF16>(o * inv);
}

template <int D, bool BF16>
__global__ __launch_bounds__((64 * waves_per_cu<D>())) void attn_sparse_kernel(Args a) {
    constexpr int NW = Dim<D>::NW, NG = Dim<D>::NG, NH = Dim<D>::NH, VD = Dim<D>::VD;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
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

    h16x8 qf[NW];
    const float factor = load_q<D, BF16>(a, row, head, hb, c, q, qf);
    f32x4 o[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) o[h] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -__builtin_inff(), l = 0.0f;
    uint8_t* region = lds + wave * region_bytes<D>();

    KTile<D> k;
    uint32_t vw[VD];
    constexpr int SW = NG * 64 / 4;            // dwords of V scales
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

    for (int first = piece * a.each + wave; first < end; first += 64 * waves) {
        // entry first + lane * waves of the list: its block, and its tile's place
        const int i = first + lane * waves;
        const int blk = i < end ? list[i] : -1;
        long long place = 0;
        bool there = blk >= 0 && blk <= at >> 6;           // at is below the table's end
        if (there) {
            const int col = blk / tiles, id = tr[col];
            there = (unsigned)id < (unsigned)a.g.n_pages;
            place = (((long long)id * a.g.kv_heads + head) * tiles + (blk - col * tiles)) * kv::tile_bytes(NG);
        }
        uint64_t todo = __ballot(there);
        if (!todo) continue;
        const int place_lo = (int)place, place_hi = (int)(place >> 32);
        auto tile_of = [&](int j) {
            return a.cache + ((long long)(uint32_t)__builtin_amdgcn_readlane(place_lo, j) |
                              (long long)__builtin_amdgcn_readlane(place_hi, j) << 32);
        };
        int j = __ffsll((unsigned long long)todo) - 1;
        {
            const uint8_t* t = tile_of(j);
            load_k<D>(k, t, c, q);
            load_v(t);
        }
        while (todo) {
            todo &= todo - 1;
            const int base = __builtin_amdgcn_readlane(blk, j) << 6;       // the tile's first position
            const int nj = todo ? __ffsll((unsigned long long)todo) - 1 : j;
            const uint8_t* nt = tile_of(nj);
            f32x4 s[4];
#pragma unroll
            for (int bl = 0; bl < 4; ++bl) {
                s[bl] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < NW; ++w) s[bl] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_frag<D>(k, bl, w), qf[w], s[bl], 0, 0, 0);
            }
            if (todo) load_k<D>(k, nt, c, q);
            if (base + 63 > at) {
                // the row's own block: what lies behind it is not seen. Its bytes may be anything, a
                // NaN scale among them, which a zero weight would let through: its scales are 0
#pragma unroll
                for (int bl = 0; bl < 4; ++bl)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (base + 16 * bl + 4 * q + e > at) s[bl][e] = -__builtin_inff();
#pragma unroll
                for (int u = 0; u < (SW + 63) / 64; ++u) {
                    const int at_byte = (u * 64 + lane) * 4;   // byte 4x + y of a group: position 16 (x % 4) + 4 (x / 4) + y
                    const int x = (at_byte & 63) >> 2;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        if (base + 16 * (x & 3) + 4 * (x >> 2) + y > at) vs[u] &= ~(255u << (8 * y));
                }
            }
            // V to LDS; this wave's earlier reads of the region are done (LDS keeps a wave's order)
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int u = 0; u < VD / 4; ++u)
                *(uint4*)(region + u * 1024 + lane * 16) = uint4{vw[4 * u], vw[4 * u + 1], vw[4 * u + 2], vw[4 * u + 3]};
#pragma unroll
            for (int u = 0; u < (SW + 63) / 64; ++u)
                if (u * 64 + lane < SW) *(uint32_t*)(region + Dim<D>::kVBytes + (u * 64 + lane) * 4) = vs[u];
            __builtin_amdgcn_wave_barrier();
            if (todo) load_v(nt);

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
                for (int h = 0; h < NH; ++h) o[h] *= alpha;
            }
            const float top = m == -__builtin_inff() ? 0.0f : m;
            h16x8 p[2];
            float add = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e >> 2][e & 3] - top, factor, kLift));
                add += x;
                p[e >> 3][e & 7] = (_Float16)x;
            }
            l += add;
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
                    const int h = 2 * g + hh, vrow = 16 * (c >> 2) + 4 * q + (c & 3);
                    const i32x2 vt = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                        (__attribute__((address_space(3))) i32x2*)(region + h * 512 + vrow * 8));
#pragma unroll
                    for (int st = 0; st < 2; ++st)
                        o[h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            decode8((uint32_t)vt[st], sv[4 * st], sv[4 * st + 1], sv[4 * st + 2], sv[4 * st + 3]), p[st], o[h], 0, 0, 0);
                }
            }
            j = nj;
        }
    }

    // join the waves: each leaves its share in LDS, then takes every waves-th column block
    l = sum_over_q(l);
    __syncthreads();
    {
        f32x4* buf = (f32x4*)(lds + wave * join_bytes<D>());
        float* ml = (float*)(buf + NH * 64);
#pragma unroll
        for (int h = 0; h < NH; ++h) buf[h * 64 + lane] = o[h];
        if (q == 0) {
            ml[c] = m;
            ml[16 + c] = l;
        }
    }
    __syncthreads();
    for (int h = wave; h < NH; h += waves) {
        float jm = -__builtin_inff(), jl = 0.0f;
        for (int w = 0; w < waves; ++w) jm = fmaxf(jm, ((const float*)(lds + w * join_bytes<D>() + NH * 1024))[c]);
        const float safe = jm == -__builtin_inff() ? 0.0f : jm;
        f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < waves; ++w) {
            const uint8_t* from = lds + w * join_bytes<D>();
            const float* ml = (const float*)(from + NH * 1024) + c;
            const float f = __builtin_amdgcn_exp2f((ml[0] - safe) * factor);
            jl = __builtin_fmaf(ml[16], f, jl);
            acc += ((const f32x4*)from)[h * 64 + lane] * f;
        }
        if (a.pieces > 1) {
            const long long slot = blockIdx.x;
            ((f32x4*)a.part)[(slot * NH + h) * 64 + lane] = acc;
            if (h == 0 && q == 0) {
                float* pm = a.part_ml + slot * 48 + c;
                pm[0] = jm;
                pm[16] = jl;
                pm[32] = factor;
            }
            continue;
        }
        store_out<D, BF16>(a, row, head, hb, h, c, q, acc, jl);
    }
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
    // Units enough for two a CU are whole, by four waves each; fewer take all the waves that
    // a CU has, and where their lists are long, several CUs.
    p.pieces = 1;
    if (p.units >= 2 * kCus) {
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
    const int per_wave = join_bytes<D>() > region_bytes<D>() ? join_bytes<D>() : region_bytes<D>();
    hipLaunchKernelGGL((attn_sparse_kernel<D, BF16>), dim3((unsigned)(p.units * p.pieces)), dim3(64 * p.waves), p.waves * per_wave, s, a);
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
