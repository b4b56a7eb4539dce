// Append to the block-scaled cache in one kernel (lrkv_append_scaled and
// lrkv_prefill_scaled): the projection on tensor cores, as in append_tc.cu, whose
// epilogue finds the scales and stores codes.
//
// A block of tokens and a head have to meet in one accumulator for that:
//  * rows: a row tile is 128 positions of one request, from a multiple of 128 on
//    (blocks of 16, 32, 64 or 128 tokens do not cross it).  Its rows of X are
//    consecutive and start at any row, even before the request's first (rows of others
//    in the tile are computed and left out).  Tiles of all requests are numbered one
//    after the other; every warp finds its own by a scan over the requests;
//  * columns: the shared rows of a group (d_h = 128) are a block of 128 columns; of the
//    private rows as many whole heads as fit in 128 columns (r = 48: two, 96).  Two
//    neighbouring blocks make a tile (S_K and S_V of a group; two of R).
// A pair of CTAs (cta_group::2) takes two row tiles by one column tile, M = 256, N = twice
// the block's width; the ring, the two accumulators and the warps' parts are append_tc.cu's.
//
// Epilogue, thread = row, four warps: the exponent that the largest magnitude of
// every head over 16 rows needs (from tensor memory), those of a block's rows through shared memory; then
// the values are read again, scaled, rounded and stored: r bytes a head and row.  Rows of
// the block that were there before are threads of the tile too: they shrink their own
// codes where the scale grows.  Where the caller wants the values in bf16 (prefill),
// they are stored beside the codes.
//
// 16,384 rows of 8 prompts, d = 2048, 16 heads, r = 48: 94 us, 63.3 at the measured bf16 peak, 123
// staged in fp32 (the projection's rows written, read again and quantised).  The issuing thread
// waits 22,000 of its 160,000 cycles for copies and 1000 for the epilogue; the rest is the
// tensor cores': 535 cycles a step of 256 x 192 x 64, whose products alone are 384, while
// shared memory serves operands and 28 KB of copies a step.  Two epilogues side by side
// (eight warps) or a seventh stage changed it by 0.3%.
#include <algorithm>

#include "append_kernels.cuh"
#include "scaled_kernels.cuh"
#include "tc_pair.cuh"

namespace lrkv {

namespace {

constexpr int kBM = 128, kBK = 64, kStages = 7;
constexpr int kABytes = kBM * kBK * 2, kBBytes = 128 * kBK * 2, kStage = kABytes + kBBytes;
constexpr int kMaxHeads = 32;  // heads of a column tile (two blocks of 128 columns, r = 8)
constexpr int kThreads = 192;  // producer, MMA, 4 epilogue warps
constexpr int kTmemCols = 512;

struct Bars {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], meet;
    uint32_t tmem;
    // of two tiles in turn: exponents that 16 rows need; old exponents of the block that has
    // rows from before (a tile has one at most)
    int8_t top[2][kMaxHeads][8];
    int8_t was[2][kMaxHeads];
};
constexpr int kOffBars = kStages * kStage;
constexpr int kSmem = kOffBars + (int)sizeof(Bars) + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

struct Maps {
    CUtensorMap x;     // X [n, d], box 64 x 128
    CUtensorMap w[4];  // W_S_K, W_S_V [G 128, d]; U_K, U_V [H r, d]: box 64 x the block's width
};

struct Args {
    ScaledPools c;
    ScaledRows rows;
    int d, clusters;
    int hb, bw, rblocks;  // heads and columns of a private block, blocks of a pool
    int per, coltiles;    // blocks of a column tile (2 or 1); tiles: of shared rows, then of private ones
    // bf16 values beside the codes (y[0] NULL: none): row b * ypages * 64 + position,
    // or (ypages 0) the cache's row
    __nv_bfloat16 *y[4];
    int ypages;
};

// One request's new rows that have a position in its page table.
struct Span {
    int b, row, pos, count;  // first row, its position, rows
    __device__ __forceinline__ int tiles() const { return count > 0 ? (pos + count - 1) / kBM - pos / kBM + 1 : 0; }
};
__device__ __forceinline__ Span span_of(const Args &a, int b, bool speaks) {
    const int r0 = a.rows.cu_rows[b], r1 = min(a.rows.cu_rows[b + 1], a.rows.n);
    Span s = {b, 0, 0, 0};
    if (r0 < 0 || r0 >= r1) return s;
    const int start = a.rows.start_pos[b];
    const int64_t max_len = (int64_t)a.rows.max_pages * a.c.page_size;
    const int64_t ra = r0 + max((int64_t)0, -(int64_t)start), rz = min((int64_t)r1, r0 + max_len - (int64_t)start);
    if (speaks && (ra > r0 || rz < r1)) status_or(a.rows.status, LRKV_STATUS_BAD_ROW);
    if (ra >= rz) return s;
    s.row = (int)ra;
    s.pos = start + ((int)ra - r0);
    s.count = (int)(rz - ra);
    return s;
}

// A row tile: 128 positions from `base` on, of the rows of a span; row `x0` of X (maybe
// negative) is the one at `base`.  b = -1: none.
struct RowTile {
    int b, base, x0, lo, hi;  // positions lo .. hi - 1 are new
};

// The requests' tiles, by a whole warp: lanes hold consecutive requests.
struct Tiles {
    int per, upto, total;  // requests a lane; tiles of its own and of the lanes before; all
    __device__ __forceinline__ Tiles(const Args &a, int lane, bool speaks) {
        per = (a.rows.B + 31) / 32;
        const int b0 = min(a.rows.B, lane * per), b1 = min(a.rows.B, b0 + per);
        upto = 0;
        // (requests that do not overlap have far fewer than 2^29 tiles; others stop there)
        constexpr int kMost = 1 << 29;
        for (int b = b0; b < b1; ++b) upto = min(upto + span_of(a, b, speaks).tiles(), kMost);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto = min(upto + v, kMost);
        }
        total = __shfl_sync(0xffffffffu, upto, 31);
    }
    __device__ __forceinline__ RowTile at(const Args &a, int t) const {
        if (t >= total) return {-1, 0, 0, 0, 0};
        const int th = __popc(__ballot_sync(0xffffffffu, upto <= t));
        int before = th > 0 ? __shfl_sync(0xffffffffu, upto, max(th - 1, 0)) : 0;
        Span s;
        for (int b = th * per;; ++b) {
            s = span_of(a, b, false);
            const int k = s.tiles();
            if (t < before + k) break;
            before += k;
        }
        const int base = (s.pos / kBM + t - before) * kBM;
        return {s.b, base, s.row + (base - s.pos), max(s.pos, base), min(s.pos + s.count, base + kBM)};
    }
};

// Column tile ct: pools and first heads of its two blocks, heads of a block, its columns and a
// head's.
struct ColTile {
    int pool[2], head[2], heads, bw, width;
};
__device__ __forceinline__ ColTile col_tile(const Args &a, int ct) {
    if (a.per == 1) {  // (one block: the first entries)
        if (ct < 2 * a.c.G) return {{ct & 1, 0}, {ct >> 1, 0}, 1, 128, 128};
        const int k = ct - 2 * a.c.G;
        return {{2 + k / a.rblocks, 0}, {k % a.rblocks * a.hb, 0}, a.hb, a.bw, a.c.r};
    }
    if (ct < a.c.G) return {{0, 1}, {ct, ct}, 1, 128, 128};
    const int k0 = 2 * (ct - a.c.G), k1 = k0 + 1;
    return {{2 + k0 / a.rblocks, 2 + k1 / a.rblocks}, {k0 % a.rblocks * a.hb, k1 % a.rblocks * a.hb}, a.hb, a.bw, a.c.r};
}

constexpr uint32_t kInfBits = 0x7f800000u;

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    append_scaled_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    Bars &bar = *reinterpret_cast<Bars *>(smem + kOffBars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_ctarank(), cluster = blockIdx.x >> 1, nk = a.d / kBK;

    if (tid == 0) {
        // (full and acc_empty are used in rank 0 only)
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&bar.acc_full[k], 1);
            mbar_init(&bar.acc_empty[k], 8);  // one arrival per epilogue warp of both CTAs
        }
        mbar_init(&bar.meet, 128);
        fence_barrier_init();
        prefetch_tensormap(&maps.x);
        for (int k = 0; k < 4; ++k) prefetch_tensormap(&maps.w[k]);
    }
    // (tensor memory is taken after the wait: a predecessor on this SM may still
    // have to take its own)
    pdl_wait();
    if (warp == 1) tmem_alloc_pair(&bar.tmem, kTmemCols);
    // both CTAs' barriers are initialised before either copies into the other
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    pdl_launch_dependents();
    bool ok = true;

    // ---- this cluster's items: (pair of row tiles, column tile), column tiles fastest
    const Tiles tiles(a, lane, warp == 2 && blockIdx.x == 0);
    const int64_t items = (int64_t)((tiles.total + 1) / 2) * a.coltiles;
    const int64_t it0 = items * cluster / a.clusters, it1 = items * (cluster + 1) / a.clusters;
    int issued = 0;  // producer: k-steps whose copies were requested

    if (warp == 0) {
        // ---- producer
        const uint32_t full0 = mapa_rank(&bar.full[0], 0);
        int s = 0, n = 0, rp = -1;
        RowTile rt = {};
        for (int64_t item = it0; item < it1 && ok; ++item) {
            const int r = (int)(item / a.coltiles);
            if (r != rp) {
                rt = tiles.at(a, 2 * r + rank);
                rp = r;
            }
            const ColTile ct = col_tile(a, (int)(item % a.coltiles));
            // this CTA's half of B: its block, or its half of the one block
            const int k = a.per == 2 ? rank : 0, brows = a.per == 2 ? ct.bw : ct.bw / 2;
            const int wrow = (k ? ct.head[1] : ct.head[0]) * ct.width + (a.per == 2 ? 0 : rank * brows);
            const CUtensorMap *wm = &maps.w[k ? ct.pool[1] : ct.pool[0]];
            const int x0 = rt.b < 0 ? a.rows.n : rt.x0;  // (no such tile: zeros)
            const uint32_t bytes = 2 * (kABytes + brows * 128);
            for (int kt = 0; kt < nk; ++kt) {
                if (n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bar.empty[s], (n - 1) & 1));
                if (!ok) break;
                if (lane == 0) {
                    uint8_t *st = smem + s * kStage;
                    const uint32_t fb = full0 + 8u * s;  // rank 0's stage barrier
                    if (rank == 0) mbar_arrive_expect_tx(&bar.full[s], bytes);
                    tma_load_2d_pair(st, &maps.x, kt * kBK, x0, fb);
                    tma_load_2d_pair(st + kABytes, wm, kt * kBK, wrow, fb);
                }
                __syncwarp();
                ++issued;
                if (++s == kStages) {
                    s = 0;
                    ++n;
                }
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---- MMA issuer (the pair's rows, M = 256)
        int s = 0, n = 0, i = 0;
        for (int64_t item = it0; item < it1 && ok; ++item, ++i) {
            const ColTile ct = col_tile(a, (int)(item % a.coltiles));
            const uint32_t idesc = tc_idesc_bf16(2 * kBM, a.per * ct.bw);
            const int acc = i & 1;
            // the epilogue has drained this accumulator's previous tile
            if (i >= 2 && !mbar_wait(&bar.acc_empty[acc], ((i >> 1) - 1) & 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + acc * 256;
            for (int kt = 0; kt < nk; ++kt) {
                if (!mbar_wait(&bar.full[s], n & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + s * kStage);
                const uint64_t ad = sw128_kmajor_desc(sa), bd = sw128_kmajor_desc(sa + kABytes);
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)  // K = 16 per instruction: +32 bytes
                    tc2_mma_f16(d, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), idesc, (kt | kk) != 0);
                tc2_commit_both(&bar.empty[s]);  // these products have read the stage
                if (++s == kStages) {
                    s = 0;
                    ++n;
                }
            }
            if (!ok) break;
            tc2_commit_both(&bar.acc_full[acc]);  // accumulator complete
        }
    } else if (warp >= 2) {
        // ---- epilogue: thread = row = tensor-memory lane of its quadrant
        const int q = warp & 3, row = 32 * q + lane, block = a.c.block, ps = a.c.page_size;
        uint32_t met = 0;
        int i = 0, rp = -1, pos = 0, bpos = 0, kept = 0;
        int64_t dr = -1, yr = -1;  // the row's place in the cache and among the bf16 values
        int64_t was_block = -1;    // the block that has rows from before
        bool fresh = false, old = false, first = false;  // a new row; one from before in a new row's block; its block's first new one
        for (int64_t item = it0; item < it1 && ok; ++item, ++i) {
            const int r = (int)(item / a.coltiles), acc = i & 1;
            if (r != rp) {  // (while the products run)
                rp = r;
                const RowTile rt = tiles.at(a, 2 * r + rank);
                auto place = [&](int p) -> int64_t {
                    const int32_t page = a.rows.page_table[(size_t)rt.b * a.rows.max_pages + p / ps];
                    return page < 0 || page >= a.c.num_pages ? -1 : (int64_t)page * ps + p % ps;
                };
                pos = rt.base + row;
                bpos = pos / block * block;  // the block's first position
                kept = rt.lo > bpos && rt.lo < bpos + block ? rt.lo - bpos : 0;  // its rows from before
                fresh = rt.b >= 0 && pos >= rt.lo && pos < rt.hi;
                old = rt.b >= 0 && pos < rt.lo && kept > 0;
                first = fresh && pos == max(bpos, rt.lo);
                dr = fresh || old ? place(pos) : -1;
                if (fresh && dr < 0) status_or(a.rows.status, LRKV_STATUS_BAD_PAGE);
                if (dr < 0) fresh = old = first = false;
                yr = !a.ypages ? dr : pos < a.ypages * 64 ? (int64_t)rt.b * a.ypages * 64 + pos : -1;
                const int64_t at = rt.b >= 0 && rt.lo % block ? place(rt.lo) : -1;
                was_block = at >= 0 ? at / block : -1;
            }
            const ColTile ct = col_tile(a, (int)(item % a.coltiles));
            const int width = ct.width, nheads = a.per * ct.heads;
            if (was_block >= 0 && row < nheads) {
                const int k = row / ct.heads, head = (k ? ct.head[1] : ct.head[0]) + row % ct.heads;
                const int pool = k ? ct.pool[1] : ct.pool[0], heads = a.c.heads(pool);
                bar.was[i & 1][row] = head < heads ? (int8_t)clamp_exp(a.c.exp[pool][was_block * heads + head]) : 0;
            }
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar.acc_full[acc], (i >> 1) & 1)))) break;
            tc_fence_after();
            const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + acc * 256;
            int8_t (*top)[8] = bar.top[i & 1];
            // ---- largest finite magnitudes of 16 rows, head by head
            uint32_t col = 0;  // (heads lie next to each other, the second block's behind the first's columns)
#pragma unroll 1
            for (int h = 0; h < nheads; ++h) {
                if (h == ct.heads) col = ct.bw;
                uint32_t m = 0;
                auto largest = [&](const uint32_t *v, int n) {
#pragma unroll
                    for (int e = 0; e < n; ++e) {
                        const uint32_t u = v[e] & 0x7fffffffu;
                        m = max(m, u < kInfBits ? u : 0u);
                    }
                };
                int c = 0;
#pragma unroll 1
                for (; c + 16 <= width; c += 16, col += 16) {
                    uint32_t v[16];
                    tmem_ld16(lanes + col, v);
                    largest(v, 16);
                }
                if (c < width) {
                    uint32_t v[8];
                    tmem_ld8(lanes + col, v);
                    largest(v, 8);
                    col += 8;
                }
                if (!fresh) m = 0;
#pragma unroll
                for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                if ((lane & 15) == 0) top[h][row >> 4] = (int8_t)needed_exp(__uint_as_float(m));
            }
            mbar_arrive(&bar.meet);
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar.meet, met++ & 1)))) break;
            // ---- scale, round, store
            col = 0;
#pragma unroll 1
            for (int h = 0; h < nheads; ++h) {
                if (h == ct.heads) col = ct.bw;
                const bool second = h >= ct.heads;
                const int pool = second ? ct.pool[1] : ct.pool[0];
                const int head = second ? ct.head[1] + h - ct.heads : ct.head[0] + h, heads = a.c.heads(pool);
                const bool live = head < heads;  // (the last block may have fewer heads)
                const int was = kept ? bar.was[i & 1][h] : LRKV_SCALED_MIN_EXP;
                int e = was;
                for (int g = 0; g < block / 16; ++g) e = max(e, (int)top[h][((bpos & (kBM - 1)) >> 4) + g]);
                if (live && first && (!kept || e > was)) a.c.exp[pool][dr / block * heads + head] = (uint8_t)(e + 127);
                const float inv = exp2i(-e), back = exp2i(e);
                const bool put = live && fresh;
                uint8_t *code = a.c.code[pool] + (dr * heads + head) * width;
                __nv_bfloat16 *y = a.y[0] && put && yr >= 0 ? a.y[pool] + (yr * heads + head) * width : nullptr;
                // eight values: their codes, and (y) what those are worth in bf16
                auto codes = [&](const uint32_t *v, uint32_t *w, uint32_t *p) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)  // (the conversion would saturate an infinity)
                        x[j] = (v[j] & 0x7fffffffu) == kInfBits ? __uint_as_float(0x7fffffffu) : __uint_as_float(v[j]) * inv;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        w[j] = (uint32_t)e4m3x2_from_f32(x[4 * j], x[4 * j + 1]) |
                               ((uint32_t)e4m3x2_from_f32(x[4 * j + 2], x[4 * j + 3]) << 16);
                    if (y) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t h2 = f16x2_from_e4m3x2((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
                            p[j] = pack_bf16(f.x * back, f.y * back);
                        }
                    }
                };
                const bool wide = width % 16 == 0;  // (then a head's codes lie at multiples of 16 bytes)
                int c = 0;
#pragma unroll 1
                for (; c + 16 <= width; c += 16, col += 16) {
                    uint32_t v[16], w[4], p[8];
                    tmem_ld16(lanes + col, v);
                    if (put) {
                        codes(v, w, p);
                        codes(v + 8, w + 2, p + 4);
                        if (wide) {
                            *reinterpret_cast<uint4 *>(code + c) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
                            *reinterpret_cast<uint2 *>(code + c) = make_uint2(w[0], w[1]);
                            *reinterpret_cast<uint2 *>(code + c + 8) = make_uint2(w[2], w[3]);
                        }
                        if (y) {
                            reinterpret_cast<uint4 *>(y + c)[0] = make_uint4(p[0], p[1], p[2], p[3]);
                            reinterpret_cast<uint4 *>(y + c)[1] = make_uint4(p[4], p[5], p[6], p[7]);
                        }
                    }
                    __syncwarp();
                }
                if (c < width) {
                    uint32_t v[8], w[2], p[4];
                    tmem_ld8(lanes + col, v);
                    col += 8;
                    if (put) {
                        codes(v, w, p);
                        *reinterpret_cast<uint2 *>(code + c) = make_uint2(w[0], w[1]);
                        if (y) *reinterpret_cast<uint4 *>(y + c) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    __syncwarp();
                }
                if (live && old && e > was) {
                    const float s = exp2i(max(was - e, -126));
                    for (int c = 0; c < width; c += 8) {
                        uint2 *p = reinterpret_cast<uint2 *>(code + c);
                        const uint2 w = *p;
                        *p = make_uint2(shrink_codes(w.x, s), shrink_codes(w.y, s));
                    }
                }
                __syncwarp();
            }
            // this warp has read its lanes of the accumulator
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(mapa_rank(&bar.acc_empty[acc], 0));
        }
    }
    if (!ok) status_or(a.rows.status, LRKV_STATUS_TIMEOUT);
    // Never leave with copies in flight into this CTA's shared memory (only
    // possible after a timeout: normally the MMA issuer consumed every stage).
    // (rank 0's stage barriers count the copies of both CTAs)
    if (warp == 0 && lane == 0 && !ok && rank == 0)
        for (int k = max(0, issued - kStages); k < issued; ++k) mbar_wait(&bar.full[k % kStages], (k / kStages) & 1);
    // neither CTA leaves while the other may still copy into it or release
    // its stages
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// [rows, d] bf16, K (= d) innermost; box 64 x `box_rows` with 128-byte swizzle.
bool map_rows(CUtensorMap *m, const void *base, int64_t rows, int d, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)d, (uint64_t)rows}, strides[1] = {(uint64_t)d * 2};
    const uint32_t box[2] = {kBK, (uint32_t)box_rows};
    return tma_map_bf16(m, base, 2, dims, strides, box);
}

// Heads of a private block: as many as fit in 128 columns, their columns a multiple of 16.
int block_heads(int r) {
    for (int hb = 128 / r; hb > 0; --hb)
        if (hb * r % 16 == 0 && 2 * hb <= kMaxHeads) return hb;
    return 0;
}

}  // namespace

bool append_scaled_tc_fits(const ScaledPools &c, int n, int B, int d) {
    // Here or staged (the projection's rows in fp32, then a write).  Tiles are 128 positions of one
    // request, so requests of few rows leave most of theirs empty: 64 of 2 rows take 47.4 us
    // here and 20 staged, 24 of 100 rows 38.7 and 33.0, 32 of 256 rows 70.4 and 68.6, 16 of
    // 20 rows 19.1 and 20.3, 4 of 512 rows 28.9 and 30.1, 8 prompts of 16,384 rows 94 and 123.
    // Two of 33 rows 15.7 and 17.3, but one of 64, where the row kernel runs, 15.4 and 12.4.
    return n > 64 && B <= 16 + n / 512 && d % kBK == 0 && c.d_h == 128 && c.r <= 128 && block_heads(c.r) > 0 && c.block <= 128 &&
           128 % c.block == 0 && tc_encode() != nullptr;
}

cudaError_t launch_append_scaled_tc(const ScaledAppendArgs &p) {
    const ScaledPools &c = p.c;
    Args a = {};
    a.c = c;
    a.rows = p.rows;
    a.d = p.d;
    a.hb = block_heads(c.r);
    a.bw = a.hb * c.r;
    a.rblocks = (c.H + a.hb - 1) / a.hb;
    // One block a tile while all of them run at once: each of twice as many SMs then does half
    // of the products and of the epilogue (512 rows: 16.0 us, 18.2 with two).  Otherwise two,
    // which need half the copies of X per product.  (N = one block's columns: a multiple of 32
    // for a pair of CTAs.)
    const int64_t pairs = (p.rows.n / kBM + 2 * (int64_t)p.rows.B + 1) / 2;
    a.per = a.bw % 32 == 0 && 2 * pairs * 2 * (c.G + a.rblocks) <= device_sm_count() ? 1 : 2;
    a.coltiles = (2 / a.per) * (c.G + a.rblocks);
    const int share = a.per == 2 ? 1 : 2;  // CTAs that share a block's rows
    a.ypages = p.ypages;
    for (int k = 0; k < 4; ++k) a.y[k] = static_cast<__nv_bfloat16 *>(p.y[k]);
    Maps maps;
    if (!map_rows(&maps.x, p.X, p.rows.n, p.d, kBM) || !map_rows(&maps.w[0], p.W_S_K, (int64_t)c.G * 128, p.d, 128 / share) ||
        !map_rows(&maps.w[1], p.W_S_V, (int64_t)c.G * 128, p.d, 128 / share) ||
        !map_rows(&maps.w[2], p.U_K, (int64_t)c.H * c.r, p.d, a.bw / share) ||
        !map_rows(&maps.w[3], p.U_V, (int64_t)c.H * c.r, p.d, a.bw / share))
        return cudaErrorInvalidValue;
    cudaError_t e = smem_limit_once(append_scaled_tc_kernel, kSmem);
    if (e != cudaSuccess) return e;
    a.clusters = (int)std::max<int64_t>(1, std::min<int64_t>(pairs * a.coltiles, device_sm_count() / 2));
    return launch_pdl(append_scaled_tc_kernel, dim3(2 * a.clusters), dim3(kThreads), kSmem, p.stream, maps, a);
}

}  // namespace lrkv
