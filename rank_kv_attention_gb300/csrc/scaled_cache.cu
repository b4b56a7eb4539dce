// Writing, reading back and laying out the block-scaled cache (lrkv_write_scaled,
// lrkv_read_scaled, and the bf16 layout that lrkv_prefill_scaled attends).
//
// value = code * 2^e: codes E4M3, one exponent per (block of tokens, head) of each
// pool, the least with which the block's largest magnitude a fits, a <= 448 * 2^e.
// Both directions move bytes and do next to nothing with them: bound by HBM for many
// rows and by dependent lookups (row -> request -> page -> block) for few.
#include <algorithm>

#include "scaled_kernels.cuh"

namespace lrkv {

namespace {

// ---------------------------------------------------------------------------
// Writing.  The unit is the rows of one call in one block: those of request b
// from its first row to the end of that row's block, then whole blocks.  Unit u
// is found without a prefix sum: number request b's first unit key(b) =
// cu_rows[b] / block + 2 b, and the unit that begins at row i after it i / block +
// 2 b + 1.  These grow strictly (a later unit's row is at least `block` further on, and
// the next request's key counts two more), so u has one owner: the last b with
// key(b) <= u.  A few u have none; there are n / block + 2 B of them.
//
// A CTA takes a slab of neighbouring heads of one pool of a unit.  A thread stays with
// one 16-byte column of it and takes every rows_par-th row, so rows are read and codes
// written whole; it holds its values in registers (8 vectors: 64 rows of a slab of
// 256 bytes), the heads' maxima meet in shared memory, and the codes go out.  Longer blocks
// are read twice, the second time out of L2.  16,384 bf16 rows of 16 heads, r = 48 take
// 18.6 us, 13.0 at the copy bandwidth: half of the time instructions issue (conversions, and what
// a CTA does for its few vectors).  One warp per head, with rows of 96 bytes, took 41; four
// vectors a thread 30.  A row each of 16 requests: 2.4, of 512: 8.9 (33 with slabs of heads for
// whole blocks).
// ---------------------------------------------------------------------------
constexpr int kWriteThreads = 128, kHeld = 8;

// n / d by a multiplication: `mul` is 2^32 / d rounded up (0: d = 1), n d below 2^32.  (A
// division by a variable is 20 to 100 instructions; with nine of them a warp took 1020 for
// its six vectors a thread.)
inline uint32_t div_mul(uint32_t d) { return d > 1 ? (uint32_t)(((uint64_t(1) << 32) + d - 1) / d) : 0; }
__device__ __forceinline__ int div_by(int n, uint32_t mul) { return mul ? (int)__umulhi((uint32_t)n, mul) : n; }
// The same by a multiple of 16 up to 1024 (tokens of a block, of a page): n below 2^30 + 2^10
inline uint32_t div16_mul(int d) { return div_mul((uint32_t)d / 16); }
__device__ __forceinline__ int div16_by(int n, uint32_t mul) { return div_by(n >> 4, mul); }

// Slabs of a pool: heads of one, and how many; 16-byte vectors of a row of it, rows that the
// threads take at a time; divisors of those and of a head's columns; of block and page.
struct Slabs {
    int heads[4], count[4], vpr[4], rows_par[4];
    uint32_t by_vpr[4], by_rows[4], by_width[4], by_block, by_page;
};

// The request of a unit, its rows [r0, r1) and its first position; b = -1: none.
struct UnitOwner {
    int b, r0, r1, start;
};

// The last b in [0, B) with cu[b] / block + 2 b <= u (whole warp).  The last probes are of
// neighbouring requests, so that their rows come with them.
__device__ __forceinline__ UnitOwner owner_of_unit(const int32_t *cu, const int32_t *start, int B, uint32_t by_block, int u,
                                                   int lane) {
    int lo = 0, hi = B;
    for (;;) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const bool in = i < hi;
        const int c0 = in ? cu[i] : 0;
        int c1 = 0, s = 0;
        if (in && step == 1) {
            c1 = cu[i + 1];
            s = start[i];
        }
        const uint32_t no = ~__ballot_sync(0xffffffffu, in && (int64_t)div16_by(max(c0, 0), by_block) + 2 * (int64_t)i <= u);
        const int k = no ? __ffs(no) - 1 : 32;  // probes that hold
        if (k == 0) return {-1, 0, 0, 0};       // (only in the first round)
        if (step == 1)
            return {lo + k - 1, __shfl_sync(0xffffffffu, c0, k - 1), __shfl_sync(0xffffffffu, c1, k - 1),
                    __shfl_sync(0xffffffffu, s, k - 1)};
        lo += (k - 1) * step;
        hi = min(hi, lo + step);
    }
}

template <typename T> struct Bits;
template <> struct Bits<__nv_bfloat16> {
    static constexpr int V = 8;  // elements of a 16-byte vector
    // largest magnitude's bits of the four words' halves, as fp32 bits
    __device__ static uint32_t top(const uint4 &v) {
        const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
        const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ static void get(const uint4 &v, float (&x)[8]) {
        x[0] = bf16lo(v.x); x[1] = bf16hi(v.x); x[2] = bf16lo(v.y); x[3] = bf16hi(v.y);
        x[4] = bf16lo(v.z); x[5] = bf16hi(v.z); x[6] = bf16lo(v.w); x[7] = bf16hi(v.w);
    }
};
template <> struct Bits<float> {
    static constexpr int V = 4;
    __device__ static uint32_t top(const uint4 &v) {
        return max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
    }
    __device__ static void get(const uint4 &v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
};

constexpr uint32_t kInf = 0x7f800000u;

// The same over a vector's finite values (0 where it has none).
template <typename T>
__device__ __forceinline__ uint32_t top_finite(const uint4 &v) {
    float x[Bits<T>::V];
    Bits<T>::get(v, x);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < Bits<T>::V; ++e) {
        const uint32_t u = __float_as_uint(x[e]) & 0x7fffffffu;
        if (u < kInf) m = max(m, u);
    }
    return m;
}

__device__ __forceinline__ uint64_t f2_mul(float lo, float hi, uint64_t s) {
    uint64_t r;
    asm("{ .reg .b64 t; mov.b64 t, {%1, %2}; mul.rn.f32x2 %0, t, %3; }" : "=l"(r) : "f"(lo), "f"(hi), "l"(s));
    return r;
}

// Codes of one vector of values times `inv`; ODD: there may be infinities (which the
// conversion would saturate) among them.
template <typename T, bool ODD>
__device__ __forceinline__ void put_codes(uint8_t *dst, const uint4 &v, float inv) {
    constexpr int V = Bits<T>::V;
    float x[V];
    Bits<T>::get(v, x);
    uint64_t s2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(inv));
    uint32_t w[V / 4];
#pragma unroll
    for (int e = 0; e < V; e += 2) {
        if (ODD)
#pragma unroll
            for (int k = e; k < e + 2; ++k)
                if ((__float_as_uint(x[k]) & 0x7fffffffu) == kInf) x[k] = __uint_as_float(0x7fffffffu);
        float lo, hi;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(f2_mul(x[e], x[e + 1], s2)));
        const uint32_t c = e4m3x2_from_f32(lo, hi);
        w[e / 4] = e % 4 ? w[e / 4] | c << 16 : c;
    }
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(dst) = w[0];
}

template <typename T>
__global__ void __launch_bounds__(kWriteThreads, 7) write_scaled_kernel(const __grid_constant__ ScaledWriteArgs a,
                                                                        const __grid_constant__ Slabs slabs) {
    constexpr int V = Bits<T>::V;
    __shared__ uint32_t tops[2][kWriteThreads];
    const ScaledPools &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, u = blockIdx.x;
    tops[0][tid] = tops[1][tid] = 0;
    __syncthreads();
    const bool speaks = blockIdx.y == 0 && tid == 0;  // flags a unit's faults
    // pool, heads h0 .. h0 + nh - 1
    int k = 0, slab = blockIdx.y;
    while (slab >= slabs.count[k]) slab -= slabs.count[k++];
    const int heads = c.heads(k), width = c.width(k), h0 = slab * slabs.heads[k], nh = min(slabs.heads[k], heads - h0);
    pdl_wait();
    pdl_launch_dependents();

    // ---- the unit's rows i0 .. i1 - 1, from position p0 on
    const UnitOwner own = owner_of_unit(a.rows.cu_rows, a.rows.start_pos, a.rows.B, slabs.by_block, u, lane);
    const int b = own.b, r0 = own.r0, r1 = min(own.r1, a.rows.n), start = own.start;
    if (b < 0 || r0 < 0 || r0 >= r1) return;
    const int64_t max_len = (int64_t)a.rows.max_pages * c.page_size;
    const int64_t ra64 = r0 + max((int64_t)0, -(int64_t)start);            // first row at a position >= 0
    const int64_t rz64 = min((int64_t)r1, r0 + max_len - (int64_t)start);  // rows past the table start here
    const int key = u - (div16_by(r0, slabs.by_block) + 2 * b);
    if (key == 0 && speaks && (ra64 > r0 || rz64 < r1)) status_or(a.rows.status, LRKV_STATUS_BAD_ROW);
    if (ra64 >= rz64) return;
    const int ra = (int)ra64, rz = (int)rz64, pa = start + (ra - r0);  // (all below 2^30 from here on)
    const int i2 = ra + (div16_by(pa, slabs.by_block) + 1) * c.block - pa;  // first row of the second unit
    int i0 = ra, i1 = i2;
    if (key > 0) {
        const int m = u - 2 * b - 1 - div16_by(i2, slabs.by_block);
        if (m < 0 || (int64_t)m * c.block >= rz - i2) return;
        i0 = i2 + m * c.block;
        i1 = i0 + c.block;
    }
    i1 = min(i1, rz);
    if (i0 >= i1) return;
    const int p0 = pa + (i0 - ra), rows = i1 - i0;

    // ---- this thread's column and rows
    const int rows_par = slabs.rows_par[k];
    const int row0 = div_by(tid, slabs.by_vpr[k]), cv = tid - row0 * slabs.vpr[k];
    const int hl = div_by(cv * V, slabs.by_width[k]);  // head in the slab (the last slab may have fewer)
    const bool active = row0 < rows_par && hl < nh;
    const int mine = active && row0 < rows ? div_by(rows - row0 + rows_par - 1, slabs.by_rows[k]) : 0;
    const int64_t ld = a.ld[k], step = ld * rows_par;
    const T *x = static_cast<const T *>(a.x[k]) + (int64_t)(i0 + row0) * ld + h0 * width + cv * V;
    uint4 val[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
        if (j < mine) val[j] = *reinterpret_cast<const uint4 *>(x + j * step);
    // (the lookups of the destination are on their way meanwhile)
    const int pi = div16_by(p0, slabs.by_page);
    const int32_t page = a.rows.page_table[(size_t)b * a.rows.max_pages + pi];
    if (page < 0 || page >= c.num_pages) {
        if (speaks) status_or(a.rows.status, LRKV_STATUS_BAD_PAGE);
        return;
    }
    const int slot = p0 - pi * c.page_size, row = page * c.page_size + slot, blk = div16_by(row, slabs.by_block);
    const int before = row - blk * c.block;  // (a block's first row is a multiple of it in the pool)
    uint8_t *eb = c.exp[k] + (int64_t)blk * heads + h0 + hl;
    const int old = before && active ? clamp_exp(*eb) : LRKV_SCALED_MIN_EXP;
    const int row_bytes = heads * width;
    uint8_t *code = c.code[k] + (int64_t)(row + row0) * row_bytes + h0 * width + cv * V;

    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
        if (j < mine) top = max(top, Bits<T>::top(val[j]));
    for (int j = kHeld; j < mine; ++j) top = max(top, Bits<T>::top(*reinterpret_cast<const uint4 *>(x + j * step)));
    if (mine) atomicMax(&tops[0][hl], top);
    // infinities or NaN in the slab: the finite values decide
    const bool odd = __syncthreads_or(top >= kInf);
    if (odd) {
        top = 0;
        for (int j = 0; j < mine; ++j) top = max(top, top_finite<T>(*reinterpret_cast<const uint4 *>(x + j * step)));
        if (mine) atomicMax(&tops[1][hl], top);
        __syncthreads();
    }
    if (!active) return;
    const int e = max(old, needed_exp(__uint_as_float(tops[odd][hl])));
    const float inv = exp2i(-e);
    const int64_t cstep = (int64_t)row_bytes * rows_par;
    if (!odd) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (j < mine) put_codes<T, false>(code + j * cstep, val[j], inv);
    }
    for (int j = odd ? 0 : kHeld; j < mine; ++j)
        put_codes<T, true>(code + j * cstep, *reinterpret_cast<const uint4 *>(x + j * step), inv);
    // ---- rows of the block before the new ones, where the scale grew
    if (before && e > old) {
        const float s = exp2i(max(old - e, -126));  // (2^-126 of any code rounds to zero too)
        uint8_t *first = code - (int64_t)before * row_bytes;
        for (int r = row0; r < before; r += rows_par, first += cstep) {
            if constexpr (V == 8) {
                uint2 *p = reinterpret_cast<uint2 *>(first);
                const uint2 w = *p;
                *p = make_uint2(shrink_codes(w.x, s), shrink_codes(w.y, s));
            } else {
                uint32_t *p = reinterpret_cast<uint32_t *>(first);
                *p = shrink_codes(*p, s);
            }
        }
    }
    if (row0 == 0 && cv * V == hl * width && (before == 0 || e > old)) *eb = (uint8_t)(e + 127);
}

// ---------------------------------------------------------------------------
// Reading.  A CTA takes a few rows; a thread takes 8 columns (which lie in one head) of all
// of them, so a warp reads 256 consecutive bytes of a row.  Bound by how many rows are on
// their way: a CTA looks its rows up (request, page, three dependent loads), meets, loads
// and stores, and others have to fill the gaps.  40,000 rows of 16 heads, r = 48 in bf16 take
// 36.2 us with 8 rows a CTA and five CTAs an SM (31.8 at the copy bandwidth), 42.4 with 16
// and two, 36.4 with 4 and eight; one request of 777 rows in fp32 3.8 with 8, 4.1 with 4.
// The layout for a prefill's attention takes 4 rows a CTA where it is short and waited for (512
// rows behind 3001: 49.3 us, 51.2 with 8), and 8 where its CTAs are many, of which those past a
// request's history only leave (8 prompts of 2048 rows: 305.1 us, 306.9 with 4).
// ---------------------------------------------------------------------------
constexpr int kReadThreads = 256, kReadRows = 8;

// Eight codes times 2^e.
__device__ __forceinline__ void widen8(const uint2 &w, float s, float (&x)[8]) {
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t h2 = f16x2_from_e4m3x2((uint16_t)(u[k >> 1] >> (16 * (k & 1))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
        x[2 * k] = f.x * s;
        x[2 * k + 1] = f.y * s;
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Of the rows of a CTA: row of the cache (-1: none), its block, row of the output;
// whether all of them lie in one block.
template <int ROWS>
struct RowSet {
    int src[ROWS], block[ROWS], dst[ROWS];
};

template <typename T, int ROWS>
__device__ __forceinline__ void copy_rows(const ScaledPools &c, const RowSet<ROWS> &set, bool one_block, void *const *y,
                                          const int64_t *ld) {
    const int chunks = (c.G * c.d_h + c.H * c.r) / 4;  // of 8 columns, in a row of all pools
    for (int ch = threadIdx.x; ch < chunks; ch += kReadThreads) {
        int k = 0, col = 8 * ch;
        while (col >= c.heads(k) * c.width(k)) {
            col -= c.heads(k) * c.width(k);
            ++k;
        }
        const int heads = c.heads(k), row_bytes = heads * c.width(k), head = col / c.width(k);
        const uint8_t *code = c.code[k] + col, *exp = c.exp[k] + head;
        T *out = static_cast<T *>(y[k]) + col;
        const int64_t ldk = ld[k];
        uint2 w[ROWS];
        int e[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (set.src[i] >= 0) w[i] = *reinterpret_cast<const uint2 *>(code + (int64_t)set.src[i] * row_bytes);
        if (one_block) {
            e[0] = exp[(int64_t)set.block[0] * heads];
#pragma unroll
            for (int i = 1; i < ROWS; ++i) e[i] = e[0];
        } else {
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                if (set.src[i] >= 0) e[i] = exp[(int64_t)set.block[i] * heads];
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (set.src[i] < 0) continue;
            float x[8];
            widen8(w[i], exp2i(clamp_exp(e[i])), x);
            store8(out + (int64_t)set.dst[i] * ldk, x);
        }
    }
}

// Pool row of position `pos` of request b, or -1.
__device__ __forceinline__ int pool_row(const ScaledPools &c, const ScaledRows &r, int b, int64_t pos) {
    if (pos < 0 || pos >= (int64_t)r.max_pages * c.page_size) {
        status_or(r.status, LRKV_STATUS_BAD_ROW);
        return -1;
    }
    const int p = (int)pos, pi = p / c.page_size;
    const int32_t page = r.page_table[(size_t)b * r.max_pages + pi];
    if (page < 0 || page >= c.num_pages) {
        status_or(r.status, LRKV_STATUS_BAD_PAGE);
        return -1;
    }
    return page * c.page_size + (p - pi * c.page_size);
}

template <typename T>
__global__ void __launch_bounds__(kReadThreads, 5) read_scaled_kernel(const __grid_constant__ ScaledReadArgs a) {
    constexpr int ROWS = kReadRows;
    __shared__ RowSet<ROWS> set;
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x < ROWS) {
        const int i = blockIdx.x * ROWS + threadIdx.x;
        int s = -1;
        if (i < a.rows.n) {
            const int b = request_of_row(a.rows.cu_rows, a.rows.B, i);
            if (b < a.rows.B && a.rows.cu_rows[b] <= i)
                s = pool_row(a.c, a.rows, b, (int64_t)a.rows.start_pos[b] + (i - a.rows.cu_rows[b]));
        }
        set.src[threadIdx.x] = s;
        set.block[threadIdx.x] = s >= 0 ? s / a.c.block : -1;
        set.dst[threadIdx.x] = i;
    }
    __syncthreads();
    const int mine = threadIdx.x < ROWS ? set.block[threadIdx.x] : set.block[0];
    const bool one = !__syncthreads_or(mine != set.block[0]) && mine >= 0;
    copy_rows<T, ROWS>(a.c, set, one, a.y, a.ld);
}

template <int ROWS>
__global__ void __launch_bounds__(kReadThreads, 5) expand_scaled_kernel(const __grid_constant__ ScaledExpandArgs a,
                                                                        int tiles) {
    __shared__ RowSet<ROWS> set;
    __shared__ int64_t ld[4];
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x / tiles, p0 = (blockIdx.x % tiles) * ROWS;
    const int r0 = a.rows.cu_rows[b], r1 = min(a.rows.cu_rows[b + 1], a.rows.n);
    const int64_t start = a.rows.start_pos[b];
    const int64_t ctx = r0 >= 0 && r0 < r1 ? min((int64_t)a.max_ctx, start + (r1 - r0)) : 0;
    const int64_t copied = a.history ? min(ctx, start) : ctx;
    // rows from max_ctx on that have a place: written, not attended
    if (p0 == 0 && threadIdx.x == 0 && r0 >= 0 && r0 < r1 &&
        max(start, (int64_t)a.max_ctx) < min(start + (r1 - r0), (int64_t)a.rows.max_pages * a.c.page_size))
        status_or(a.rows.status, LRKV_STATUS_BAD_SEQLEN);
    if (p0 >= copied && !(a.table && p0 % 64 == 0)) return;
    if (threadIdx.x < 4) ld[threadIdx.x] = (int64_t)a.c.heads(threadIdx.x) * a.c.width(threadIdx.x);
    if (threadIdx.x < ROWS) {
        const int p = p0 + threadIdx.x;
        const int s = p < ctx ? pool_row(a.c, a.rows, b, p) : -1;
        set.src[threadIdx.x] = p < copied ? s : -1;
        set.block[threadIdx.x] = p < copied && s >= 0 ? s / a.c.block : -1;
        set.dst[threadIdx.x] = a.table ? b * a.pages * 64 + p : s;
        // (a cache page holds whole pages of 64 rows: one is missing where its first row is)
        if (a.table && threadIdx.x == 0 && p0 % 64 == 0) a.table[(size_t)b * a.pages + p0 / 64] = s >= 0 ? b * a.pages + p0 / 64 : -1;
    }
    __syncthreads();
    const int mine = threadIdx.x < ROWS ? set.block[threadIdx.x] : set.block[0];
    const bool one = !__syncthreads_or(mine != set.block[0]) && mine >= 0;
    if (p0 >= copied) return;
    copy_rows<__nv_bfloat16, ROWS>(a.c, set, one, a.y, ld);
}

}  // namespace

cudaError_t launch_write_scaled(const ScaledWriteArgs &a) {
    const int64_t units = a.rows.n / a.c.block + 2 * (int64_t)a.rows.B;
    const int V = a.f32 ? 4 : 8;
    // columns of a slab: a vector a thread, fewer where a unit (of a block, or of twice a request's rows
    // on average) is longer than the values that threads hold then (and one head at least)
    const int rows = (int)std::min<int64_t>(a.c.block, 2 * ((a.rows.n + (int64_t)a.rows.B - 1) / a.rows.B));
    const int vecs = std::max(1, std::min(kWriteThreads, kWriteThreads * kHeld / rows));
    Slabs slabs;
    int total = 0;
    for (int k = 0; k < 4; ++k) {
        const int heads = a.c.heads(k), each = std::max(1, vecs / (a.c.width(k) / V));
        const int parts = (heads + each - 1) / each;
        slabs.heads[k] = (heads + parts - 1) / parts;
        slabs.count[k] = (heads + slabs.heads[k] - 1) / slabs.heads[k];
        slabs.vpr[k] = slabs.heads[k] * a.c.width(k) / V;
        slabs.rows_par[k] = kWriteThreads / slabs.vpr[k];
        slabs.by_vpr[k] = div_mul(slabs.vpr[k]);
        slabs.by_rows[k] = div_mul(slabs.rows_par[k]);
        slabs.by_width[k] = div_mul(a.c.width(k));
        total += slabs.count[k];
    }
    slabs.by_block = div16_mul(a.c.block);
    slabs.by_page = div16_mul(a.c.page_size);
    const dim3 grid((unsigned)units, total);
    return a.f32 ? launch_pdl(write_scaled_kernel<float>, grid, dim3(kWriteThreads), 0, a.stream, a, slabs)
                 : launch_pdl(write_scaled_kernel<__nv_bfloat16>, grid, dim3(kWriteThreads), 0, a.stream, a, slabs);
}

template <typename T>
static cudaError_t launch_read(const ScaledReadArgs &a) {
    return launch_pdl(read_scaled_kernel<T>, dim3((a.rows.n + kReadRows - 1) / kReadRows), dim3(kReadThreads), 0, a.stream, a);
}

cudaError_t launch_read_scaled(const ScaledReadArgs &a) {
    return a.f32 ? launch_read<float>(a) : launch_read<__nv_bfloat16>(a);
}

template <int ROWS>
static cudaError_t launch_expand(const ScaledExpandArgs &a) {
    const int tiles = (a.max_ctx + ROWS - 1) / ROWS;
    return launch_pdl(expand_scaled_kernel<ROWS>, dim3((unsigned)(a.rows.B * (int64_t)tiles)), dim3(kReadThreads), 0,
                      a.stream, a, tiles);
}

cudaError_t launch_expand_scaled(const ScaledExpandArgs &a) {
    // (eight CTAs of 4 rows on every SM)
    return (int64_t)a.rows.B * a.max_ctx < 32 * (int64_t)device_sm_count() ? launch_expand<4>(a) : launch_expand<8>(a);
}

}  // namespace lrkv
