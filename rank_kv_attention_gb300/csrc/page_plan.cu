// Page plan of one serving step: which pages each request gains, which pages
// no later query can see, and where every new row goes.
//
// For request b with L rows and n new ones (n = -1: the request ends):
//   gains     pages ceil(L / ps) .. ceil((L + n) / ps) - 1, taken off the end
//             of the free list in (request, page) order;
//   releases  the pages that leave the window: a query at position t sees
//             j > t - W and j < K, so page p is out of sight of every query at
//             a position >= L once (p + 1) ps <= L - W + 1 and p ps >= K, that
//             is for ceil(K / ps) <= p < D(L) = floor((L - W + 1) / ps); a step
//             from L to L + n releases the pages between max(D(L), sp) and
//             max(D(L + n), sp), sp = ceil(K / ps).  A request that ends
//             releases all that it holds.
// Released ids are appended behind what the step leaves of the free list, so
// the step's own attention, which still sees some of them, runs before any
// later step can hand them out.
//
// One launch.  Each block scans all requests itself (two passes of block scans over
// tiles of kTile requests: the lengths are a few kilobytes in L2) and writes
// its share of every tile's rows, table entries and released ids, so nothing
// waits on another block and nothing is kept between launches.  What bounds it:
// launch latency and the two scans for decode-sized steps, the 12 bytes per
// row written for large ones.  In a graph: 64 requests with a new row each 10.2 us,
// 1500 requests with 730,000 new rows 14.3 us (9.1 MB: 1.3 us at the copy
// bandwidth).
#include <algorithm>

#include "page_kernels.cuh"

namespace lrkv {

namespace {

constexpr int kNT = 512;            // threads per block
constexpr int kPer = 4;             // requests per thread and tile
constexpr int kTile = kNT * kPer;
constexpr int kRun = 4;             // rows per lane and search

// What the step does to one request.
struct Step {
    int32_t L, rows, need;  // rows it has, gains; pages it gains
    int32_t lo, hi, front;  // releases [0, front) and [lo, hi)
    bool bad, refused, ends;
    __device__ __forceinline__ int32_t released() const { return front + hi - lo; }
};

struct Geometry {
    int32_t ps, room, window, sp;
    __device__ __forceinline__ int32_t pages(int32_t n) const { return (n + ps - 1) / ps; }
    __device__ __forceinline__ int32_t dead(int32_t L) const {
        if (window == 0) return 0;
        const int32_t x = L - window + 1;
        return max(sp, x > 0 ? x / ps : 0);
    }
};

// Exclusive block scans of N sequences of kPer values per thread; totals in sum.
template <typename V, int N>
__device__ __forceinline__ void block_scan(V (&v)[N][kPer], V (&part)[N][kNT / 32], V (&sum)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    V incl[N], run[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        run[n] = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const V x = v[n][k];
            v[n][k] = run[n];
            run[n] += x;
        }
        incl[n] = run[n];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const V y = __shfl_up_sync(0xffffffffu, incl[n], o);
            if (lane >= o) incl[n] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int n = 0; n < N; ++n) part[n][warp] = incl[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        // every warp scans the warps' totals itself
        V t = lane < kNT / 32 ? part[n][lane] : 0;
#pragma unroll
        for (int o = 1; o < kNT / 32; o <<= 1) {
            const V y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        sum[n] = __shfl_sync(0xffffffffu, t, kNT / 32 - 1);
        const V before = __shfl_sync(0xffffffffu, t, warp ? warp - 1 : 0);
        const V base = incl[n] - run[n] + (warp ? before : 0);
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[n][k] += base;
    }
    __syncthreads();  // part is reused by the next scan
}

// First entry of the nondecreasing off[0 .. n] (off[0] <= x < off[n]) whose
// successor exceeds x.
__device__ __forceinline__ int find(const int32_t *off, int n, int32_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (off[mid + 1] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

struct Shared {
    int64_t part64[2][kNT / 32];
    int32_t part32[3][kNT / 32];
    // of the current tile, exclusive, with the tile's total at the end
    int32_t rows[kTile + 1], need[kTile + 1], rel[kTile + 1];
    int32_t len[kTile], lo[kTile], front[kTile];
};

}  // namespace

__global__ void __launch_bounds__(kNT) page_plan_kernel(const PagePlanArgs a) {
    extern __shared__ __align__(16) uint8_t sm_raw[];
    Shared &sm = *reinterpret_cast<Shared *>(sm_raw);
    const int tid = threadIdx.x, g = blockIdx.x, G = gridDim.x;
    pdl_wait();
    pdl_launch_dependents();
    Geometry geo;
    geo.ps = a.page_size;
    geo.room = a.max_pages * a.page_size;
    geo.window = a.window;
    geo.sp = a.window ? geo.pages(min(a.sinks, geo.room)) : 0;
    const int32_t n_in = *a.n_free;
    const int32_t n_free = min(max(n_in, 0), a.num_pages);
    uint32_t flags = n_in != n_free ? LRKV_STATUS_BAD_PAGE : 0u;

    // the next page off the end of the free list (-1 for an id that is none)
    auto fresh = [&](int32_t k) -> int32_t {
        const int32_t id = a.free_pages[n_free - 1 - k];
        return id >= 0 && id < a.num_pages ? id : -1;
    };
    // pages the step takes in all: known after one tile, or after a pass over all
    int32_t taken = 0;
    const int ntile = (a.B + kTile - 1) / kTile;
    for (int pass = ntile > 1 ? 0 : 1; pass < 2; ++pass) {
        int64_t want0 = 0, need0 = 0;          // asked for by the tiles before
        int32_t rows0 = 0, alloc0 = 0, rel0 = 0;  // granted and released by them
        for (int t0 = 0; t0 < a.B; t0 += kTile) {
            const int nb = min(kTile, a.B - t0);
            Step st[kPer];
            int64_t asked[2][kPer], asked_all[2];  // rows, pages
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = tid * kPer + k;
                Step &s = st[k];
                s.bad = s.ends = false;
                s.L = s.rows = s.need = 0;
                if (i < nb) {
                    s.L = a.seq_lens[t0 + i];
                    const int32_t n = a.new_rows[t0 + i];
                    s.bad = s.L < 0 || s.L > geo.room || n < -1 || n > geo.room - s.L;
                    s.ends = !s.bad && n == -1;
                    s.rows = s.bad || n < 0 ? 0 : n;
                    s.need = s.rows ? geo.pages(s.L + s.rows) - geo.pages(s.L) : 0;
                }
                asked[0][k] = s.rows;
                asked[1][k] = s.need;
            }
            block_scan(asked, sm.part64, asked_all);
            int32_t got[3][kPer], got_all[3];  // rows, pages, released
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                Step &s = st[k];
                const bool fits = want0 + asked[0][k] + s.rows <= a.max_rows &&
                                  (s.need == 0 || need0 + asked[1][k] + s.need <= n_free);
                s.refused = !fits && s.rows > 0;
                if (s.refused) s.rows = s.need = 0;
                s.front = 0;
                s.lo = s.hi = 0;
                if (s.ends) {
                    const int32_t held = geo.pages(s.L);
                    s.front = min(geo.sp, held);
                    s.lo = geo.dead(s.L);
                    s.hi = max(held, s.lo);
                } else if (s.rows > 0) {
                    s.lo = geo.dead(s.L);
                    s.hi = geo.dead(s.L + s.rows);
                }
                got[0][k] = s.rows;
                got[1][k] = s.need;
                got[2][k] = s.released();
            }
            block_scan(got, sm.part32, got_all);
            const int32_t rows_all = got_all[0], alloc_all = got_all[1], rel_all = got_all[2];
            want0 += asked_all[0];
            need0 += asked_all[1];
            if (pass == 0) {
                taken += alloc_all;
                continue;
            }
            if (ntile == 1) taken = alloc_all;
            const int32_t left = n_free - taken;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = tid * kPer + k;
                if (i < nb) {
                    const Step &s = st[k];
                    sm.rows[i] = got[0][k];
                    sm.need[i] = got[1][k];
                    sm.rel[i] = got[2][k];
                    sm.len[i] = s.L;
                    sm.lo[i] = s.lo;
                    sm.front[i] = s.front;
                    if (g == 0) {
                        a.seq_lens_out[t0 + i] = s.ends ? 0 : s.L + s.rows;
                        a.cu_rows[t0 + i] = rows0 + got[0][k];
                        if (s.bad) flags |= LRKV_STATUS_BAD_SEQLEN;
                        if (s.refused) flags |= LRKV_STATUS_NO_PAGES;
                    }
                }
            }
            if (tid == 0) {
                sm.rows[nb] = rows_all;
                sm.need[nb] = alloc_all;
                sm.rel[nb] = rel_all;
            }
            __syncthreads();
            // page p of the tile's request i: an entry of the table, or one of
            // the pages that it gains in this step
            auto page_of = [&](int i, int32_t p) -> int32_t {
                const int32_t held = geo.pages(sm.len[i]);
                if (p >= held) return fresh(alloc0 + sm.need[i] + p - held);
                const int32_t id = a.page_table[(size_t)(t0 + i) * a.max_pages + p];
                return id >= 0 && id < a.num_pages ? id : -1;
            };
            for (int x = g * kNT + tid; x < alloc_all; x += G * kNT) {
                const int i = find(sm.need, nb, x);
                const int32_t id = fresh(alloc0 + x);
                if (id < 0) flags |= LRKV_STATUS_BAD_PAGE;
                a.page_table[(size_t)(t0 + i) * a.max_pages + geo.pages(sm.len[i]) + x - sm.need[i]] = id;
            }
            for (int x = g * kNT + tid; x < rel_all; x += G * kNT) {
                const int i = find(sm.rel, nb, x);
                const int32_t y = x - sm.rel[i];
                const int32_t p = y < sm.front[i] ? y : sm.lo[i] + y - sm.front[i];
                const int32_t id = page_of(i, p);
                const int32_t at = left + rel0 + x;
                if (id < 0 || at >= a.num_pages) flags |= LRKV_STATUS_BAD_PAGE;
                if (at < a.num_pages) a.free_out[at] = id;
            }
            // rows: a warp takes kRun x 32 consecutive ones, a search for the first
            // of each lane and steps from there, all page ids in flight at once
            for (int x0 = (g * (kNT / 32) + (tid >> 5)) * 32 * kRun; x0 < rows_all; x0 += G * kNT * kRun) {
                int i = find(sm.rows, nb, min(x0 + (tid & 31), rows_all - 1));
                int req[kRun], pos[kRun], id[kRun];
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    const int x = min(x0 + 32 * k + (tid & 31), rows_all - 1);
                    while (sm.rows[i + 1] <= x) ++i;
                    req[k] = i;
                    pos[k] = sm.len[i] + x - sm.rows[i];
                    id[k] = page_of(i, pos[k] / geo.ps);
                }
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    const int x = x0 + 32 * k + (tid & 31);
                    if (x < rows_all) {
                        if (id[k] < 0) flags |= LRKV_STATUS_BAD_PAGE;
                        a.positions[rows0 + x] = pos[k];
                        a.seq_ids[rows0 + x] = t0 + req[k];
                        a.slots[rows0 + x] = id[k] < 0 ? -1 : id[k] * geo.ps + pos[k] % geo.ps;
                    }
                }
            }
            rows0 += rows_all;
            alloc0 += alloc_all;
            rel0 += rel_all;
            __syncthreads();  // the tile's arrays are rewritten
        }
        if (pass == 0) continue;
        const int32_t left = n_free - taken;
        for (int x = g * kNT + tid; x < left; x += G * kNT) a.free_out[x] = a.free_pages[x];
        for (int x = rows0 + g * kNT + tid; x < a.max_rows; x += G * kNT)
            a.positions[x] = a.seq_ids[x] = a.slots[x] = -1;
        if (g == 0 && tid == 0) {
            a.cu_rows[a.B] = rows0;
            *a.n_free_out = min(a.num_pages, left + rel0);
        }
    }
    if (flags) status_or(a.status, flags);
}

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s) {
    const int64_t items = (int64_t)a.max_rows + a.num_pages;
    const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), (items + 4095) / 4096));
    const cudaError_t e = smem_limit_once(page_plan_kernel, (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
    return launch_pdl(page_plan_kernel, dim3(blocks), dim3(kNT), sizeof(Shared), s, a);
}

}  // namespace lrkv
