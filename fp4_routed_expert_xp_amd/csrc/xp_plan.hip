// xp_plan.hip — who gets which pages and which place each new token takes, on the GPU:
// page tables and slot maps of a step from request lengths, and pages given back.
//
// Free pages are a stack. Sequences are served in order, so who is served follows from
// two running sums (rows and pages), which one workgroup forms, 1,024 sequences a
// round; a sequence's new pages are consecutive entries of the stack. There is no
// arithmetic to speak of: both calls are bound by the chain lengths -> sums -> stack ->
// table -> maps, a round trip to memory each (64 sequences that ask for a token each, and
// their release: 14.9 us; 150 prompts of up to 1,900 rows and 900 single tokens, and their
// release, three launches: 18.3).
#include "xp_kv_dev.h"

namespace xp {
namespace plan {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kOwnPages = 4;       // pages that a sequence's own thread moves
constexpr int kGroup = 16;         // lanes that move a longer run, four entries each at a time (a wave each: 20.5 us of 18.3)
// Up to so many rows, and kThreads sequences, the maps are the same workgroup's: a plan and its release take
// 7.2 us for some tens of rows and 8.7 with a launch of the maps' own, 9.3 and 10.2 at 2,400 rows, 10.3 and
// 10.6 at 4,700, 17.8 and 10.5 at 16,500.
constexpr int kOneLaunchRows = 4096;
constexpr int kMaxRows = 1 << 24;

struct Step {
    const int32_t* lens;
    const int32_t* want;
    int32_t* table;
    const int32_t* free_pages;
    int32_t* free_count;
    int32_t* cu;
    int32_t* start;
    int32_t* lens_out;
    int32_t* seq;
    int32_t* pos;
    long long* slot;
    int batch, max_pages, page, n_pages, rows;
};

// Columns of a table that n positions take: n is at most 2^31 - 1025.
__device__ __forceinline__ int columns_of(int n, int page) { return (int)(((unsigned)n + (unsigned)page - 1) / (unsigned)page); }

__device__ __forceinline__ int stack_height(const int32_t* count, int n_pages) {
    const int n = count[0];
    return n < 0 ? 0 : (n > n_pages ? n_pages : n);
}

// One row's entries of the maps; b: its sequence.
__device__ __forceinline__ void put_row(const Step& a, int r, int b, int first) {
    const int at = a.start[b] + (r - first), col = at / a.page;
    const int id = a.table[(long long)b * a.max_pages + col];
    a.seq[r] = b;
    a.pos[r] = at;
    a.slot[r] = (unsigned)id < (unsigned)a.n_pages ? (long long)id * a.page + (at - col * a.page) : -1ll;
}
__device__ __forceinline__ void put_none(const Step& a, int r) {
    a.seq[r] = -1;
    a.pos[r] = -1;
    a.slot[r] = -1;
}

struct Run {
    int b, col, n, base;   // n entries of sequence b's table from col on; the stack's entry behind base others
};

__global__ __launch_bounds__(kThreads) void plan_kernel(Step a, int maps) {
    __shared__ long long part_r[kWaves];
    __shared__ int part_p[kWaves];
    __shared__ Run runs[kThreads];
    __shared__ int ends[kThreads];
    __shared__ int n_runs, all_rows, all_pages;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int height = stack_height(a.free_count, a.n_pages);
    const long long cap = (long long)a.max_pages * a.page;
    long long before_r = 0, before_p = 0;      // asked for by earlier rounds' sequences
    if (tid == 0) all_rows = all_pages = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + tid;
        const bool in = b < a.batch;
        const int len = in ? a.lens[b] : 0, want = in ? a.want[b] : 0;
        const bool asks = want > 0 && len >= 0 && (long long)len + want <= cap;
        // more rows than there is room for: one too many says it, and keeps a wave's sum in 32 bits
        const int r = asks ? (want > a.rows ? a.rows + 1 : want) : 0;
        const int col = asks ? columns_of(len, a.page) : 0;
        const int p = asks && want <= a.rows ? columns_of(len + want, a.page) - col : 0;
        const int sum_r = wave_incl_sum(r), sum_p = wave_incl_sum(p);
        if (lane == 63) {
            part_r[wave] = sum_r;
            part_p[wave] = sum_p;
        }
        if (tid == 0) n_runs = 0;
        __syncthreads();
        long long upto_r = before_r + sum_r, upto_p = before_p + sum_p;
        for (int w = 0; w < kWaves; ++w) {
            const long long x = part_r[w];
            const int y = part_p[w];
            upto_r += w < wave ? x : 0;
            upto_p += w < wave ? y : 0;
            before_r += x;
            before_p += y;
        }
        // both sums only grow: who does not fit, and everyone behind, is not served
        const bool fits = in && upto_r <= a.rows && upto_p <= height;
        const uint64_t served = __ballot(fits);
        if (served && lane == 63 - __builtin_clzll(served)) {
            atomicMax(&all_rows, (int)upto_r);
            atomicMax(&all_pages, (int)upto_p);
        }
        if (fits && p > 0) {
            int32_t* t = a.table + (long long)b * a.max_pages + col;
            const int base = (int)upto_p - p;
            if (p <= kOwnPages)
                for (int j = 0; j < p; ++j) t[j] = a.free_pages[height - 1 - (base + j)];
            else
                runs[atomicAdd(&n_runs, 1)] = Run{b, col, p, base};
        }
        __syncthreads();
        if (in) {
            const int end = fits ? (int)upto_r : all_rows;
            a.start[b] = len;
            a.lens_out[b] = fits ? len + r : len;
            a.cu[b + 1] = end;
            ends[tid] = end;                   // of use where there is one round
        }
        for (int i = tid / kGroup; i < n_runs; i += kThreads / kGroup) {
            const Run u = runs[i];
            int32_t* t = a.table + (long long)u.b * a.max_pages + u.col;
            for (int j0 = tid % kGroup; j0 < u.n; j0 += 4 * kGroup) {
                int id[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) id[k] = j0 + k * kGroup < u.n ? a.free_pages[height - 1 - (u.base + j0 + k * kGroup)] : 0;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (j0 + k * kGroup < u.n) t[j0 + k * kGroup] = id[k];
            }
        }
        __syncthreads();
    }
    if (tid == 0) {
        a.cu[0] = 0;
        a.free_count[0] = height - all_pages;
    }
    if (!maps) return;
    for (int r = tid; r < a.rows; r += kThreads) {
        if (r >= all_rows) {
            put_none(a, r);
            continue;
        }
        int lo = 0, hi = a.batch - 1;          // the first sequence that ends behind r
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (ends[mid] > r)
                hi = mid;
            else
                lo = mid + 1;
        }
        put_row(a, r, lo, lo ? ends[lo - 1] : 0);
    }
}

// The maps of many rows or sequences: a wave finds the sequences of its first and last
// row, its lanes search between them.
__global__ __launch_bounds__(256) void map_kernel(Step a) {
    const int lane = threadIdx.x & 63, first = (blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 64;
    if (first >= a.rows) return;
    const int r = first + lane, last = first + 63 < a.rows ? first + 63 : a.rows - 1;
    int lo = kv::sequence_of_row(a.cu, a.batch, first), hi = kv::sequence_of_row(a.cu, a.batch, last);
    if (r >= a.rows) return;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > r)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (lo < a.batch)
        put_row(a, r, lo, a.cu[lo]);
    else
        put_none(a, r);
}

// No sequences: no row anywhere, in the arrays that are there.
__global__ __launch_bounds__(256) void none_kernel(Step a) {
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r == 0 && a.cu) a.cu[0] = 0;
    if (r >= a.rows) return;
    if (a.seq) a.seq[r] = -1;
    if (a.pos) a.pos[r] = -1;
    if (a.slot) a.slot[r] = -1;
}

struct Release {
    const int32_t* lens;
    const int32_t* keep;
    int32_t* table;
    int32_t* free_pages;
    int32_t* free_count;
    int batch, max_pages, page, n_pages;
};

// From the last sequence to the first, and in each from its last page to the first, so
// that the pages of a plan come to lie as they were: an entry's place is the number of
// pages behind it.
__global__ __launch_bounds__(kThreads) void release_kernel(Release a) {
    __shared__ int part[kWaves];
    __shared__ Run runs[kThreads];
    __shared__ int found[kThreads];
    __shared__ int n_runs;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cap = a.max_pages * a.page;
    const auto is_page = [&](int id) { return (unsigned)id < (unsigned)a.n_pages; };
    long long at = stack_height(a.free_count, a.n_pages);
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = a.batch - 1 - (b0 + tid);
        int col = 0, n = 0;
        if (b >= 0) {
            const int len = a.lens[b] > cap ? cap : a.lens[b], keep = a.keep[b] < 0 ? 0 : a.keep[b];
            if (len > keep) {
                col = columns_of(keep, a.page);
                n = columns_of(len, a.page) - col;
            }
        }
        int32_t* t = a.table + (long long)(b < 0 ? 0 : b) * a.max_pages + col;
        const bool own = n <= kOwnPages;
        if (tid == 0) n_runs = 0;
        __syncthreads();
        int ids[kOwnPages], pages = 0;
        if (own) {
#pragma unroll
            for (int j = 0; j < kOwnPages; ++j) {
                ids[j] = j < n ? t[j] : -1;
                pages += is_page(ids[j]);
            }
        } else {
            runs[atomicAdd(&n_runs, 1)] = Run{b, col, n, tid};
        }
        __syncthreads();
        for (int i = tid / kGroup; i < n_runs; i += kThreads / kGroup) {
            const Run u = runs[i];
            const int32_t* ut = a.table + (long long)u.b * a.max_pages + u.col;
            int c = 0;
#pragma unroll 4
            for (int j = tid % kGroup; j < u.n; j += kGroup) c += is_page(ut[j]);
#pragma unroll
            for (int k = 1; k < kGroup; k <<= 1) c += __shfl_xor(c, k);
            if (tid % kGroup == 0) found[u.base] = c;
        }
        __syncthreads();
        if (!own) pages = found[tid];
        // below 2^31 where no page is named twice; where the sum wraps, nothing is put outside the stack
        const int sum = wave_incl_sum(pages);
        if (lane == 63) part[wave] = sum;
        __syncthreads();
        long long to = at + sum - pages;       // where this sequence's last page goes
        for (int w = 0; w < kWaves; ++w) {
            to += w < wave ? part[w] : 0;
            at += part[w];
        }
        if (own) {
#pragma unroll
            for (int j = kOwnPages - 1; j >= 0; --j)
                if (j < n) {
                    if (is_page(ids[j])) {
                        if ((unsigned long long)to < (unsigned long long)a.n_pages) a.free_pages[to] = ids[j];
                        ++to;
                    }
                    t[j] = -1;
                }
        } else {
            found[tid] = to < 0 || to > a.n_pages ? a.n_pages : (int)to;   // entries from n_pages on are not kept
        }
        __syncthreads();
        for (int i = tid / kGroup; i < n_runs; i += kThreads / kGroup) {
            const Run u = runs[i];
            int32_t* ut = a.table + (long long)u.b * a.max_pages + u.col;
            long long put = found[u.base];
            for (int j0 = u.n - 1 - tid % kGroup; j0 + tid % kGroup >= 0; j0 -= 4 * kGroup) {
                int id[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) id[k] = j0 - k * kGroup >= 0 ? ut[j0 - k * kGroup] : -1;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // the pages of the group's lanes, this one's place among them
                    const uint32_t there = (uint32_t)(__ballot(is_page(id[k])) >> (lane & ~(kGroup - 1))) & ((1u << kGroup) - 1);
                    const long long mine = put + __popc(there & ((1u << (tid % kGroup)) - 1));
                    if (is_page(id[k]) && mine < a.n_pages) a.free_pages[mine] = id[k];
                    if (j0 - k * kGroup >= 0) ut[j0 - k * kGroup] = -1;
                    put += __popc(there);
                }
            }
        }
        __syncthreads();
    }
    if (tid == 0) a.free_count[0] = at < 0 || at > a.n_pages ? a.n_pages : (int)at;
}

// Whether any written array shares a byte with another one (host).
struct Span {
    const void* p;
    int64_t bytes;
    bool written;
};
static bool overlap(const Span* s, int n) {
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < i; ++j) {
            if (!s[i].p || !s[j].p || (!s[i].written && !s[j].written)) continue;
            const uintptr_t a = (uintptr_t)s[i].p, b = (uintptr_t)s[j].p;
            if (s[i].bytes > 0 && s[j].bytes > 0 && a < b + s[j].bytes && b < a + s[i].bytes) return true;
        }
    return false;
}

}  // namespace plan
}  // namespace xp

using namespace xp;
using namespace xp::plan;

XP_API int xp_kv_plan(const xp_kv_dims* dims, int32_t batch, int32_t max_pages, int32_t rows, const int32_t* lens,
                      const int32_t* want, int32_t* table, const int32_t* free_pages, int32_t* free_count, int32_t* cu_rows,
                      int32_t* start, int32_t* lens_out, int32_t* row_seq, int32_t* row_pos, int64_t* row_slot, void* stream) {
    const int st = kv::check_geo(dims, batch, max_pages);
    if (st != XP_OK) return st;
    if (rows < 0 || rows > kMaxRows) return XP_ERR_SHAPE;
    hipStream_t s = (hipStream_t)stream;
    const int64_t b4 = 4 * (int64_t)batch, r4 = 4 * (int64_t)rows;
    if (batch == 0) {
        const Span spans[] = {{cu_rows, 4, true}, {row_seq, r4, true}, {row_pos, r4, true}, {row_slot, 2 * r4, true}};
        for (const Span& x : spans)
            if (!kv::aligned_to(x.p, x.p == row_slot ? 8 : 4)) return XP_ERR_SHAPE;
        if (overlap(spans, (int)(sizeof(spans) / sizeof(spans[0])))) return XP_ERR_SHAPE;
        if (!cu_rows && (rows == 0 || (!row_seq && !row_pos && !row_slot))) return XP_OK;
        Step a{};
        a.cu = cu_rows;
        a.seq = row_seq;
        a.pos = row_pos;
        a.slot = (long long*)row_slot;
        a.rows = rows;
        hipLaunchKernelGGL(none_kernel, dim3(rows ? (unsigned)((rows + 255) / 256) : 1u), dim3(256), 0, s, a);
        return launch_status();
    }
    if (!lens || !want || !table || !free_pages || !free_count || !cu_rows || !start || !lens_out ||
        (rows > 0 && (!row_seq || !row_pos || !row_slot)))
        return XP_ERR_NULL;
    const Span spans[] = {{lens, lens == lens_out ? 0 : b4, false}, {want, b4, false}, {table, b4 * max_pages, true},
                          {free_pages, 4 * (int64_t)dims->n_pages, false}, {free_count, 4, true}, {cu_rows, b4 + 4, true},
                          {start, b4, true}, {lens_out, b4, true}, {row_seq, r4, true}, {row_pos, r4, true}, {row_slot, 2 * r4, true}};
    for (const Span& x : spans)
        if (!kv::aligned_to(x.p, 4)) return XP_ERR_SHAPE;
    if (!kv::aligned_to(row_slot, 8) || overlap(spans, (int)(sizeof(spans) / sizeof(spans[0])))) return XP_ERR_SHAPE;
    const Step a{lens, want, table, free_pages, free_count, cu_rows, start, lens_out, row_seq, row_pos, (long long*)row_slot,
                 batch, max_pages, dims->page, dims->n_pages, rows};
    const bool one = batch <= kThreads && rows <= kOneLaunchRows;
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kThreads), 0, s, a, one ? 1 : 0);
    const int rc = launch_status();
    if (rc != XP_OK || one || rows == 0) return rc;
    hipLaunchKernelGGL(map_kernel, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0, s, a);
    return launch_status();
}

XP_API int xp_kv_release(const xp_kv_dims* dims, int32_t batch, int32_t max_pages, const int32_t* lens, const int32_t* keep,
                         int32_t* table, int32_t* free_pages, int32_t* free_count, void* stream) {
    const int st = kv::check_geo(dims, batch, max_pages);
    if (st != XP_OK) return st;
    if (batch == 0) return XP_OK;
    if (!lens || !keep || !table || !free_pages || !free_count) return XP_ERR_NULL;
    const int64_t b4 = 4 * (int64_t)batch;
    const Span spans[] = {{lens, b4, false}, {keep, b4, false}, {table, b4 * max_pages, true},
                          {free_pages, 4 * (int64_t)dims->n_pages, true}, {free_count, 4, true}};
    for (const Span& s : spans)
        if (!kv::aligned_to(s.p, 4)) return XP_ERR_SHAPE;
    if (overlap(spans, (int)(sizeof(spans) / sizeof(spans[0])))) return XP_ERR_SHAPE;
    const Release a{lens, keep, table, free_pages, free_count, batch, max_pages, dims->page, dims->n_pages};
    hipLaunchKernelGGL(release_kernel, dim3(1), dim3(kThreads), 0, (hipStream_t)stream, a);
    return launch_status();
}
