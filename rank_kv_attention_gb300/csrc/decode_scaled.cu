// Decode over the block-scaled cache on tensor cores (lrkv_decode_scaled), the
// codes multiplied as they are.
//
//   x_j = (2^eSK q.S_K[j] + 2^eRK[h] p.R_K[h,j]) / sqrt(d_h),   p = q B_K[h]
//   o   = sum_j a_j 2^eSV S_V[j] + (sum_j a_j 2^eRV[h] R_V[h,j]) B_V[h]^T,  a = softmax(x)
// (reading note "Low-Rank Key Value Attention", equations 6 and 7, on E4M3 codes
// and scale exponents; d_h = 128, one shared basis).
//
// A cache tile as it lies in memory, 128 tokens x 128 bytes, is the A operand of
// tcgen05.mma kind::f8f6f4: for scores with tokens as rows (K-major), for values
// with tokens as the contraction (MN-major).  So no code is ever widened: the
// copies go to shared memory by TMA and from there into the tensor core, and what
// is computed per token is its scores.  The B operands are small and made here:
//  * q and p as three E4M3 terms each, x = s (t1 + t2 / 2^4 + t3 / 2^9) with s a power
//    of two that brings the largest |x| into (224, 448]: off by at most 2^-14 of x
//    or 2^-26 of the largest;
//  * the weights as two, w = t1 + t2 / 2^4, the tile's largest 256: off by at most
//    2^-9 of w (bf16's half step is 2^-8) or 2^-22 of the largest.
// Columns of one MMA are (head, term).  128 columns of R hold several heads' private
// rows; the score operand of such a box has zeros in the columns of other heads,
// and of its value products each row of D is read for its own head only.  (A NaN
// code therefore reaches the heads that share its box.)  The tensor core works
// N = 16 to 64 columns of M = 128, bound by reading A: 32 cycles per 4 KB, where HBM
// delivers 4 KB per SM in 170.
//
// Scales: a token's exponent enters its score, x + e, before the exponential: the
// value products take 2^(x + eS - MS) and 2^(x + eR - MR), each relative to the tile's
// largest per head, so tokens of loud and quiet blocks keep their precision next
// to each other.  Sums, maxima and the accumulators over tiles are fp32 in registers.
//
// Work: the requests' rows in units of 64 tokens, laid end to end and cut evenly
// over one CTA per SM; a CTA walks its tiles (two units of one request, or one).
// Each piece of a request in a CTA leaves a state in the workspace, and a second
// kernel merges and expands them by B_V[h].  A first, small kernel makes the q and p
// operands (and the offsets that the merge needs), while the first tiles are on
// their way.
//
// 11 warps: 0-3 scores and weights (thread = token = tensor-memory lane), 4-7 value
// accumulators (thread = column), 8 copies cache tiles, 9 issues the MMAs, 10 copies
// operands.  Order of the stream: keys of tile i + 1, then values of tile i, so a
// tile's softmax runs while the next keys arrive.
#include <algorithm>

#include "scaled_kernels.cuh"
#include "tc_common.cuh"

namespace lrkv {

namespace {

constexpr int kUnit = 64, kTile = 128;
constexpr int kStageBytes = kTile * 128;
constexpr int kMaxBoxes = 16, kMaxStages = 12;
constexpr int kThreads = 352;
constexpr int kSmemMost = 232448;

// Layout of one shape: the R columns in boxes of 128, which heads they hold, and
// where operands and accumulators lie.
struct Shape {
    int H, r, boxes, stages;
    int img_bytes;             // operand image of a request: q rows, p rows, factors
    int qrows, prows;          // rows (128 bytes) of the q part and of all p boxes
    int wrows;                 // rows of one weight operand
    int tmem_cols;
    uint16_t h0[kMaxBoxes];    // first head of a box
    uint16_t n[kMaxBoxes];     // score columns of a box: (head - h0) * 4 + term
    uint16_t prow[kMaxBoxes];  // its first row in the p part
    uint16_t scol[kMaxBoxes];  // its first score column
    uint16_t ha[kMaxBoxes];    // value products: first head, a multiple of 4
    uint16_t nv[kMaxBoxes];    // value columns: (head - ha) * 2 + term
    uint16_t vcol[kMaxBoxes];
    uint16_t v0, nv0;          // the shared rows' value columns
};

inline bool make_shape(int H, int r, Shape &s) {
    if (H % 4 || H < 4 || H > 32 || r % 8 || r < 8 || r > 64) return false;
    s.H = H;
    s.r = r;
    s.boxes = (H * r + 127) / 128;
    if (s.boxes > kMaxBoxes) return false;
    s.qrows = (4 * H + 15) / 16 * 16;
    int row = 0, col = s.qrows;
    for (int t = 0; t < s.boxes; ++t) {
        const int a = 128 * t / r, z = std::min(H - 1, (128 * t + 127) / r);
        s.h0[t] = (uint16_t)a;
        s.n[t] = (uint16_t)((4 * (z - a + 1) + 15) / 16 * 16);
        s.prow[t] = (uint16_t)row;
        s.scol[t] = (uint16_t)col;
        row += s.n[t];
        col += s.n[t];
    }
    s.prows = row;
    s.v0 = (uint16_t)col;
    s.nv0 = (uint16_t)((2 * H + 15) / 16 * 16);
    col += s.nv0;
    for (int t = 0; t < s.boxes; ++t) {
        const int z = std::min(H - 1, (128 * t + 127) / r);
        s.ha[t] = (uint16_t)(s.h0[t] & ~3);
        s.nv[t] = (uint16_t)((2 * (z - s.ha[t] + 1) + 15) / 16 * 16);
        s.vcol[t] = (uint16_t)col;
        col += s.nv[t];
        if (s.n[t] > 256 || s.nv[t] > 32) return false;
    }
    if (col > 512) return false;
    s.tmem_cols = 32;
    while (s.tmem_cols < col) s.tmem_cols *= 2;
    s.img_bytes = (s.qrows + s.prows) * 128 + 8 * H;
    s.wrows = 2 * H + 32;  // (a box's window may reach past the last head)
    return true;
}

// Shared memory after the ring of stages.
struct Offsets {
    int img, weights, red, fac, bars, bytes;
    __host__ __device__ explicit Offsets(const Shape &s) {
        img = s.stages * kStageBytes;
        const int one = (s.img_bytes + 1023) / 1024 * 1024;
        weights = img + 2 * one;
        red = weights + 2 * s.wrows * 128;  // [2][4][H][4 warps]: maxima, sums of the weights
        fac = red + 2 * 4 * 32 * 4 * 4;     // [2][3][H]: alpha, shared and private factor
        bars = fac + 2 * 3 * 32 * 4;
        bytes = bars + 512 + 1024;
    }
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t img_full[2], img_empty[2];
    uint64_t sc_full, sc_empty, w_full, pv_done, v_empty;
    uint64_t meet;  // of the 128 softmax threads
    uint32_t tmem;
    int first_b, first_unit, units;
    int warp_sum[kThreads / 32];
};
static_assert(sizeof(Bars) <= 512, "barriers");

struct Maps {
    CUtensorMap k[2], v[2];  // S_K, R_K; S_V, R_V: [rows][bytes], box 128 bytes x box_rows
};

struct Args {
    ScaledPools c;
    const int32_t *seq_lens, *page_table;
    const uint8_t *img;  // operand images [B][img_bytes rounded up to 256]
    int64_t img_stride;
    ScaledStates st;
    int32_t *status;
    int B, max_pages, max_len, box_rows;
};

__device__ __forceinline__ int units_of(int L, int max_len) {
    return L >= 1 && L <= max_len ? (L + kUnit - 1) / kUnit : 0;
}

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// D (+)= A B^T, 8-bit E4M3 operands in shared memory, K = 32.
__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 da, db; setp.ne.u32 p, %4, 0; mov.b64 da, {%1, %5}; "
        "mov.b64 db, {%2, %5}; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p; }" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(kSw128DescHi)
        : "memory");
}
// kind::f8f6f4, E4M3 operands, fp32 D, M = 128; B K-major; A K-major or (amn) MN-major.
__device__ __forceinline__ uint32_t idesc_f8(int N, bool amn) {
    return (1u << 4) | (amn ? 1u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&v)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Code of x (|x| <= 448) and what it leaves.
__device__ __forceinline__ uint8_t take_code(float &x) {
    const uint8_t c = (uint8_t)(e4m3x2_from_f32(x, 0.f) & 0xffu);
    x -= e4m3_to_f32(c);
    return c;
}

// Byte `k` of row `n` of an operand with 128-byte rows, as a 128-byte swizzle has it.
__device__ __forceinline__ uint32_t op_byte(int n, int k) {
    return (uint32_t)(n * 128 + ((((k >> 4) ^ n) & 7) << 4) + (k & 15));
}

// ---------------------------------------------------------------------------
// Operands: block (h, b) makes the terms of q[b, h] and p = q B_K[h] and the factors
// that bring a tile's sums to log2 units; one more block the unit offsets.
// ---------------------------------------------------------------------------
struct PrepArgs {
    const __nv_bfloat16 *q, *B_K;
    const int32_t *seq_lens;
    uint8_t *img;
    int64_t img_stride;
    int32_t *off;
    int B, max_len;
    float scale_log2;
};

__global__ void __launch_bounds__(128) scaled_prep_kernel(const __grid_constant__ PrepArgs P,
                                                          const __grid_constant__ Shape S) {
    __shared__ float qs[128], ps[64], part[128 * 8];
    __shared__ float red[8];
    __shared__ int sums[128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == (unsigned)P.B) {  // offsets, by the blocks' one column that exists for them
        if (blockIdx.y) return;
        const int per = (P.B + 127) / 128, b0 = tid * per, b1 = min(P.B, b0 + per);
        int n = 0;
        for (int b = b0; b < b1; ++b) n += units_of(P.seq_lens[b], P.max_len);
        sums[tid] = n;
        __syncthreads();
        int at = 0;
        for (int i = 0; i < tid; ++i) at += sums[i];
        for (int b = b0; b < b1; ++b) {
            P.off[b] = at;
            at += units_of(P.seq_lens[b], P.max_len);
        }
        if (b1 == P.B && b0 < b1) P.off[P.B] = at;
        return;
    }
    const int b = blockIdx.x, h = blockIdx.y, r = S.r;
    const __nv_bfloat16 *B = P.B_K + (size_t)h * 128 * r;
    qs[tid] = __bfloat162float(P.q[((size_t)b * S.H + h) * 128 + tid]);
    __syncthreads();
    // p: groups of r / 8 threads take every `parts`-th channel
    const int v8 = r / 8, parts = 128 / v8, pt = tid / v8, vc = tid % v8;
    if (pt < parts) {
        float acc[8] = {};
#pragma unroll 4
        for (int d = pt; d < 128; d += parts) {
            float y[8];
            Vec16<__nv_bfloat16>::load(B + (size_t)d * r + 8 * vc, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(qs[d], y[e], acc[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) part[(pt * v8 + vc) * 8 + e] = acc[e];
    }
    __syncthreads();
    if (tid < r) {
        float s = 0.f;
        for (int i = 0; i < parts; ++i) s += part[i * r + tid];
        ps[tid] = s;
    }
    __syncthreads();
    float mq = fabsf(qs[tid]), mp = tid < r ? fabsf(ps[tid]) : 0.f;
    // (a NaN or an infinity: the maximum says nothing, the factor carries it)
    const bool odd = !(mq <= 3.4e38f) || !(mp <= 3.4e38f);
    mq = warp_max(mq);
    mp = warp_max(mp);
    if (lane == 0) {
        red[warp] = mq;
        red[4 + warp] = mp;
    }
    const bool bad = __syncthreads_or(odd);
    const int eq = bad ? 0 : needed_exp(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const int ep = bad ? 0 : needed_exp(fmaxf(fmaxf(red[4], red[5]), fmaxf(red[6], red[7])));
    uint8_t *img = P.img + b * P.img_stride;
    {
        float x = bad ? 0.f : qs[tid] * exp2i(-eq);
        img[op_byte(4 * h, tid)] = take_code(x);
        x *= 16.f;
        img[op_byte(4 * h + 1, tid)] = take_code(x);
        x *= 32.f;
        img[op_byte(4 * h + 2, tid)] = take_code(x);
    }
    for (int t = h * r / 128; t <= (h * r + r - 1) / 128; ++t) {
        const int k = 128 * t + tid - h * r, n = 4 * (h - S.h0[t]);
        uint8_t *box = img + (S.qrows + S.prow[t]) * 128;
        float x = k >= 0 && k < r && !bad ? ps[k] * exp2i(-ep) : 0.f;
        box[op_byte(n, tid)] = take_code(x);
        x *= 16.f;
        box[op_byte(n + 1, tid)] = take_code(x);
        x *= 32.f;
        box[op_byte(n + 2, tid)] = take_code(x);
    }
    if (tid == 0) {
        float *f = reinterpret_cast<float *>(img + (S.qrows + S.prows) * 128);
        f[h] = bad ? __uint_as_float(0x7fffffffu) : P.scale_log2 * exp2i(eq);
        f[S.H + h] = P.scale_log2 * exp2i(ep);
    }
}

// ---------------------------------------------------------------------------
// One CTA's tiles, in order; every role walks them by itself.
// ---------------------------------------------------------------------------
struct Walk {
    int b, L, tok, left, seg;  // left: units of the CTA from this tile on
    __device__ Walk(const Args &a, const Bars &bar) {
        b = bar.first_b;
        left = bar.units;
        seg = 0;
        L = left ? a.seq_lens[b] : 0;
        tok = bar.first_unit * kUnit;
    }
    __device__ bool live() const { return left > 0; }
    __device__ int rows() const { return min(min(kTile, L - tok), left * kUnit); }
    __device__ bool ends() const { return tok + kTile >= L || left * kUnit <= kTile; }  // of its request here
    __device__ void next(const Args &a) {
        left -= (rows() + kUnit - 1) / kUnit;
        tok += kTile;
        if (left > 0 && tok >= L) {
            do L = a.seq_lens[++b];
            while (units_of(L, a.max_len) == 0);
            tok = 0;
            ++seg;
        }
    }
};

template <int HM>
__global__ void __launch_bounds__(kThreads, 1)
    decode_scaled_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a,
                         const __grid_constant__ Shape S) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const Offsets off(S);
    Bars &bar = *reinterpret_cast<Bars *>(smem + off.bars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = S.H, stages = S.stages, NB = S.boxes;
    const int img_stride = (S.img_bytes + 1023) / 1024 * 1024;

    // ---- this CTA's share
    {
        const int per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
        int n = 0;
        for (int b = b0; b < b1; ++b) n += units_of(a.seq_lens[b], a.max_len);
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) bar.warp_sum[warp] = inc;
        if (tid == 0) {
            for (int s = 0; s < stages; ++s) {
                mbar_init(&bar.full[s], 1);
                mbar_init(&bar.empty[s], 1);
            }
            for (int k = 0; k < 2; ++k) {
                mbar_init(&bar.img_full[k], 1);
                mbar_init(&bar.img_empty[k], 129);
            }
            mbar_init(&bar.meet, 128);
            mbar_init(&bar.sc_full, 1);
            mbar_init(&bar.sc_empty, 128);
            mbar_init(&bar.w_full, 128);
            mbar_init(&bar.pv_done, 1);
            mbar_init(&bar.v_empty, 128);
            fence_barrier_init();
            bar.first_b = 0;
            bar.first_unit = 0;
        }
        __syncthreads();
        int64_t total = 0, before = inc - n;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += bar.warp_sum[w];
            total += bar.warp_sum[w];
        }
        // (CTAs past the last unit have none, so that no request's CTAs have a gap)
        const int64_t ctas = max((int64_t)1, min((int64_t)gridDim.x, total)), g = min((int64_t)blockIdx.x, ctas);
        const int64_t u0 = total * g / ctas, u1 = min(total, total * (g + 1) / ctas);
        if (tid == 0) bar.units = (int)(u1 - u0);
        if (n && u0 >= before && u0 < before + n) {
            int64_t at = before;
            for (int b = b0; b < b1; ++b) {
                const int k = units_of(a.seq_lens[b], a.max_len);
                if (u0 < at + k) {
                    bar.first_b = b;
                    bar.first_unit = (int)(u0 - at);
                    break;
                }
                at += k;
            }
        }
    }
    if (warp == 8) tmem_alloc(&bar.tmem, S.tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    pdl_launch_dependents();
    bool ok = true;
    Walk w(a, bar);

    if (warp == 8) {
        // ================= cache tiles =================
        // lane k holds the pool row of the tile's k-th box row group (past every row,
        // which reads as zeros, where its page is none)
        const int R = a.box_rows, none = a.c.num_pages * a.c.page_size;
        auto lookup = [&](const Walk &t) {
            const int at = t.tok + lane * R;
            int row = none;
            if (lane * R < t.rows()) {
                const int32_t page = a.page_table[(size_t)t.b * a.max_pages + at / a.c.page_size];
                if (page < 0 || page >= a.c.num_pages) status_or(a.status, LRKV_STATUS_BAD_PAGE);
                else row = page * a.c.page_size + at % a.c.page_size;
            }
            return row;
        };
        int it = 0;
        auto send = [&](const CUtensorMap *m, int rows, int row) {  // the keys or values of one tile
            const int groups = (rows + R - 1) / R;
            for (int t = 0; t <= NB; ++t, ++it) {
                const int s = it % stages;
                if (it >= stages) ok = __all_sync(0xffffffffu, mbar_wait(&bar.empty[s], ((it / stages) - 1) & 1)) && ok;
                if (!ok) return;
                if (lane == 0) mbar_arrive_expect_tx(&bar.full[s], groups * R * 128);
                __syncwarp();
                // (each lane issues its own group's copy)
                if (lane < groups)
                    tma_load_2d(smem + s * kStageBytes + lane * R * 128, &m[t > 0], t > 0 ? 128 * (t - 1) : 0, row, &bar.full[s]);
            }
        };
        if (w.live()) {
            int rows = w.rows(), row = lookup(w);
            send(maps.k, rows, row);
            while (ok && w.live()) {
                w.next(a);
                int nrows = 0, nrow = none;
                if (w.live()) {
                    nrows = w.rows();
                    nrow = lookup(w);
                    send(maps.k, nrows, nrow);
                }
                if (ok) send(maps.v, rows, row);
                rows = nrows;
                row = nrow;
            }
        }
        // nothing leaves with copies in flight (the MMA issuer has waited for all unless it gave up)
        if (!ok && lane == 0)
            for (int k = max(0, it - stages); k < it; ++k) mbar_wait(&bar.full[k % stages], (k / stages) & 1);
    } else if (warp == 10) {
        // ================= operand images =================
        if (lane == 0) {
            pdl_wait();
            int last = -1;
            for (; ok && w.live(); w.next(a)) {
                if (w.seg == last) continue;
                const int s = last = w.seg, k = s & 1;
                if (s >= 2 && !mbar_wait(&bar.img_empty[k], ((s >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&bar.img_full[k], S.img_bytes);
                bulk_load(smem + off.img + k * img_stride, a.img + w.b * a.img_stride, S.img_bytes, &bar.img_full[k]);
            }
            for (int s = max(0, last - 1); s <= last; ++s) mbar_wait(&bar.img_full[s & 1], (s >> 1) & 1);
        }
    } else if (warp == 9) {
        // ================= MMA issuer =================
        const uint32_t base = smem_u32(smem);
        int it = 0, i = 0;
        auto stage_wait = [&]() {
            const bool got = __all_sync(0xffffffffu, mbar_wait(&bar.full[it % stages], (it / stages) & 1));
            tc_fence_after();
            return got;
        };
        auto keys = [&](const Walk &t, bool first) -> bool {
            const uint32_t img = base + off.img + (t.seg & 1) * img_stride;
            if (first && !__all_sync(0xffffffffu, mbar_wait(&bar.img_full[t.seg & 1], (t.seg >> 1) & 1))) return false;
            if (i > 0 && !__all_sync(0xffffffffu, mbar_wait(&bar.sc_empty, (i - 1) & 1))) return false;
            tc_fence_after();
            for (int x = 0; x <= NB; ++x, ++it) {
                if (!stage_wait()) return false;
                const uint32_t al = sw128_desc_lo(base + (it % stages) * kStageBytes, 16);
                const uint32_t bl = sw128_desc_lo(img + (x ? S.qrows + S.prow[x - 1] : 0) * 128, 16);
                const uint32_t d = tmem + (x ? S.scol[x - 1] : 0), id = idesc_f8(x ? S.n[x - 1] : S.qrows, false);
                const int steps = x ? min(4, (H * S.r - 128 * (x - 1) + 31) / 32) : 4;
                if (lane == 0) {
                    for (int k = 0; k < steps; ++k) tc_mma_f8(d, al + 2 * k, bl + 2 * k, id, k != 0);
                    tc_commit(&bar.empty[it % stages]);
                }
                __syncwarp();
            }
            if (lane == 0) {
                tc_commit(&bar.sc_full);
                if (t.ends()) tc_commit(&bar.img_empty[t.seg & 1]);
            }
            __syncwarp();
            return true;
        };
        auto values = [&](int rows, int n) -> bool {  // of the n-th tile
            if (!__all_sync(0xffffffffu, mbar_wait(&bar.w_full, n & 1))) return false;
            if (n > 0 && !__all_sync(0xffffffffu, mbar_wait(&bar.v_empty, (n - 1) & 1))) return false;
            tc_fence_after();
            const int steps = (rows + 31) / 32;
            for (int x = 0; x <= NB; ++x, ++it) {
                if (!stage_wait()) return false;
                uint8_t *st = smem + (it % stages) * kStageBytes;
                if (rows & 31) {
                    // rows past the end, of whatever bits, in the last group of 32: their
                    // weights are zero, and zero times a NaN is not
                    for (int u = rows * 8 + lane; u < steps * 32 * 8; u += 32)
                        *reinterpret_cast<uint4 *>(st + u * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const uint32_t al = sw128_desc_lo(base + (it % stages) * kStageBytes, 16);
                const uint32_t bl = sw128_desc_lo(
                    base + off.weights + (x ? S.wrows + 2 * S.ha[x - 1] : 0) * 128, 16);
                const uint32_t d = tmem + (x ? S.vcol[x - 1] : S.v0), id = idesc_f8(x ? S.nv[x - 1] : S.nv0, true);
                if (lane == 0) {
                    // 32 tokens an instruction: 32 rows of 128 bytes of A, 32 bytes of B's rows
                    for (int k = 0; k < steps; ++k) tc_mma_f8(d, al + 256 * k, bl + 2 * k, id, k != 0);
                    tc_commit(&bar.empty[it % stages]);
                }
                __syncwarp();
            }
            if (lane == 0) tc_commit(&bar.pv_done);
            __syncwarp();
            return true;
        };
        if (w.live()) {
            int rows = w.rows(), seg = w.seg;
            ok = keys(w, true);
            while (ok && w.live()) {
                w.next(a);
                int nrows = 0;
                ++i;
                if (w.live()) {
                    nrows = w.rows();
                    ok = keys(w, w.seg != seg);
                    seg = w.seg;
                }
                if (ok) ok = values(rows, i - 1);
                rows = nrows;
            }
        }
        if (!ok && lane == 0) status_or(a.status, LRKV_STATUS_TIMEOUT);
    } else if (warp < 4) {
        // ================= scores and weights: thread = token =================
        const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
        float m[HM], l[HM];
        int last = -1, nb = a.c.page_size / a.c.block;
        uint32_t met = 0;
        auto meet = [&]() -> bool {  // all four warps (a wait with a limit, as every wait here)
            mbar_arrive(&bar.meet);
            return __all_sync(0xffffffffu, mbar_wait(&bar.meet, met++ & 1));
        };
        for (int i = 0; ok && w.live(); ++i, w.next(a)) {
            // the token's scale exponents
            const int pos = w.tok + tid;
            bool there = tid < w.rows();
            int e_sk = 0, e_sv = 0;
            uint32_t e_rk[HM / 4] = {}, e_rv[HM / 4] = {};
            if (there) {
                const int32_t page = a.page_table[(size_t)w.b * a.max_pages + pos / a.c.page_size];
                there = page >= 0 && page < a.c.num_pages;
                if (there) {
                    const int64_t eb = (int64_t)page * nb + pos % a.c.page_size / a.c.block;
                    e_sk = a.c.exp[0][eb];
                    e_sv = a.c.exp[1][eb];
                    const uint32_t *rk = reinterpret_cast<const uint32_t *>(a.c.exp[2] + eb * H);
                    const uint32_t *rv = reinterpret_cast<const uint32_t *>(a.c.exp[3] + eb * H);
#pragma unroll
                    for (int k = 0; k < HM / 4; ++k)
                        if (4 * k < H) {
                            e_rk[k] = rk[k];
                            e_rv[k] = rv[k];
                        }
                }
            }
            const bool first = w.seg != last, ends = w.ends();
            last = w.seg;
            if (first) {
#pragma unroll
                for (int h = 0; h < HM; ++h) {
                    m[h] = -INFINITY;
                    l[h] = 0.f;
                }
                ok = __all_sync(0xffffffffu, mbar_wait(&bar.img_full[w.seg & 1], (w.seg >> 1) & 1));
                if (!ok) break;
            }
            const float *f = reinterpret_cast<const float *>(smem + off.img + (w.seg & 1) * img_stride +
                                                             (S.qrows + S.prows) * 128);
            ok = __all_sync(0xffffffffu, mbar_wait(&bar.sc_full, i & 1));
            if (!ok) break;
            tc_fence_after();
            float x[HM];
            const float sk = exp2i(clamp_exp(e_sk));
#pragma unroll
            for (int h = 0; h < HM; ++h) {
                if (h < H) {
                    const int ta = h * S.r / 128, tb = (h * S.r + S.r - 1) / 128;
                    uint32_t vs[4], va[4], vb[4];
                    tmem_ld4(lanes + 4 * h, vs);
                    tmem_ld4(lanes + S.scol[ta] + 4 * (h - S.h0[ta]), va);
                    if (tb != ta) tmem_ld4(lanes + S.scol[tb], vb);  // (the first head of that box)
                    tmem_wait_ld();
                    const float s = __uint_as_float(vs[0]) + (__uint_as_float(vs[1]) * 0.0625f + __uint_as_float(vs[2]) * 0.001953125f);
                    float t = __uint_as_float(va[0]) + (__uint_as_float(va[1]) * 0.0625f + __uint_as_float(va[2]) * 0.001953125f);
                    if (tb != ta)
                        t += __uint_as_float(vb[0]) + (__uint_as_float(vb[1]) * 0.0625f + __uint_as_float(vb[2]) * 0.001953125f);
                    const float rk = exp2i(clamp_exp((e_rk[h / 4] >> (8 * (h & 3))) & 0xff));
                    x[h] = there ? s * (f[h] * sk) + t * (f[H + h] * rk) : -INFINITY;
                }
            }
            tc_fence_before();
            mbar_arrive(&bar.sc_empty);
            if (ends) mbar_arrive(&bar.img_empty[w.seg & 1]);  // (the factors were read)
            // (two buffers in turn: a warp writes the one after next only when all have met again)
            float *red = reinterpret_cast<float *>(smem + off.red) + (i & 1) * 4 * 32 * 4;
            const float es = (float)clamp_exp(e_sv);
            float mine[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < HM; ++h)
                if (h < H) {
                    const float er = (float)clamp_exp((e_rv[h / 4] >> (8 * (h & 3))) & 0xff);
                    const float m0 = warp_max(x[h]), m1 = warp_max(x[h] + es), m2 = warp_max(x[h] + er);
                    if (lane == (h & 31)) {
                        mine[0] = m0;
                        mine[1] = m1;
                        mine[2] = m2;
                    }
                }
            if (lane < H)
#pragma unroll
                for (int k = 0; k < 3; ++k) red[(k * 32 + lane) * 4 + warp] = mine[k];
            ok = meet();
            // the operand of the tile before has been read
            if (ok && i > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bar.pv_done, (i - 1) & 1));
            if (!ok) break;
            float *fac = reinterpret_cast<float *>(smem + off.fac) + (i & 1) * 3 * 32;
            uint8_t *ws = smem + off.weights, *wr = ws + S.wrows * 128;
#pragma unroll
            for (int h = 0; h < HM; ++h)
                if (h < H) {
                    const float er = (float)clamp_exp((e_rv[h / 4] >> (8 * (h & 3))) & 0xff);
                    float M[3];
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const float4 v = *reinterpret_cast<const float4 *>(&red[(k * 32 + h) * 4]);
                        M[k] = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
                    }
                    const float mn = fmaxf(m[h], M[0]), ref = mn == -INFINITY ? 0.f : mn;
                    const float ms = M[1] == -INFINITY ? 0.f : M[1], mr = M[2] == -INFINITY ? 0.f : M[2];
                    const float alpha = ex2f(m[h] - ref);
                    m[h] = mn;
                    l[h] = l[h] * alpha + ex2f(x[h] - ref);
                    if (tid == h) {
                        fac[h] = alpha;
                        fac[32 + h] = ex2f(ms - ref - 8.f);
                        fac[64 + h] = ex2f(mr - ref - 8.f);
                    }
                    float y = ex2f(x[h] + es - ms + 8.f), z = ex2f(x[h] + er - mr + 8.f);
                    ws[op_byte(2 * h, tid)] = take_code(y);
                    wr[op_byte(2 * h, tid)] = take_code(z);
                    y *= 16.f;
                    z *= 16.f;
                    ws[op_byte(2 * h + 1, tid)] = take_code(y);
                    wr[op_byte(2 * h + 1, tid)] = take_code(z);
                }
            fence_proxy_async_smem();
            mbar_arrive(&bar.w_full);
            if (ends) {
                // the sums of all tokens: over the warp, then over the four warps
                float sum = 0.f;
#pragma unroll
                for (int h = 0; h < HM; ++h)
                    if (h < H) {
                        float v = l[h];
#pragma unroll
                        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                        if (lane == (h & 31)) sum = v;
                    }
                if (lane < H) red[(3 * 32 + lane) * 4 + warp] = sum;
                float *ml = a.st.ml + ((int64_t)w.b + blockIdx.x) * H * 2;
                if (!(ok = meet())) break;
#pragma unroll
                for (int h = 0; h < HM; ++h)
                    if (h < H && tid == h) {
                        const float4 v = *reinterpret_cast<const float4 *>(&red[(3 * 32 + h) * 4]);
                        ml[2 * h] = m[h];
                        ml[2 * h + 1] = (v.x + v.y) + (v.z + v.w);
                    }
            }
        }
        if (!ok && lane == 0) status_or(a.status, LRKV_STATUS_TIMEOUT);
    } else {
        // ================= value accumulators: thread = column =================
        const int col = tid - 128;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float as[HM], ar[kMaxBoxes];
        int last = -1;
        for (int i = 0; ok && w.live(); ++i, w.next(a)) {
            if (w.seg != last) {
#pragma unroll
                for (int h = 0; h < HM; ++h) as[h] = 0.f;
#pragma unroll
                for (int t = 0; t < kMaxBoxes; ++t) ar[t] = 0.f;
                last = w.seg;
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&bar.w_full, i & 1) && mbar_wait(&bar.pv_done, i & 1));
            if (!ok) break;
            tc_fence_after();
            const float *fac = reinterpret_cast<const float *>(smem + off.fac) + (i & 1) * 3 * 32;
#pragma unroll
            for (int g = 0; g < HM / 8; ++g)
                if (8 * g < H) {
                    uint32_t v[16];
                    tmem_ld16(lanes + S.v0 + 16 * g, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int h = 8 * g + k;
                        if (h < H)
                            as[h] = as[h] * fac[h] +
                                    (__uint_as_float(v[2 * k]) + __uint_as_float(v[2 * k + 1]) * 0.0625f) * fac[32 + h];
                    }
                }
#pragma unroll
            for (int t = 0; t < kMaxBoxes; ++t)
                if (t < NB) {
                    const int h = min((128 * t + col) / S.r, H - 1), k = h - S.ha[t];
                    float y = 0.f;
#pragma unroll
                    for (int g = 0; g < 2; ++g)
                        if (16 * g < S.nv[t]) {
                            uint32_t v[16];
                            tmem_ld16(lanes + S.vcol[t] + 16 * g, v);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (k == 8 * g + j) y = __uint_as_float(v[2 * j]) + __uint_as_float(v[2 * j + 1]) * 0.0625f;
                        }
                    ar[t] = ar[t] * fac[h] + y * fac[64 + h];
                }
            tc_fence_before();
            mbar_arrive(&bar.v_empty);
            if (w.ends()) {
                float *acc = a.st.acc + ((int64_t)w.b + blockIdx.x) * H * (128 + S.r);
#pragma unroll
                for (int h = 0; h < HM; ++h)
                    if (h < H) acc[h * 128 + col] = as[h];
#pragma unroll
                for (int t = 0; t < kMaxBoxes; ++t)
                    if (t < NB && 128 * t + col < H * S.r) acc[H * 128 + 128 * t + col] = ar[t];
            }
        }
        if (!ok && lane == 0) status_or(a.status, LRKV_STATUS_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, S.tmem_cols);
    }
}

// [rows][bytes] 8-bit codes; box 128 bytes x box_rows, 128-byte swizzle, zeros outside.
bool map_codes(CUtensorMap *m, const void *base, int64_t rows, int bytes, int box_rows) {
    TcEncodeFn enc = tc_encode();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)bytes};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace: unit offsets, operand images, states of up to B + CTAs pieces.
struct Ws {
    int32_t *off;
    uint8_t *img;
    int64_t img_stride;
    void *states;
    size_t bytes;
};
Ws layout(void *base, const Shape &s, int B, int ctas, int d_h) {
    Ws w;
    char *p = static_cast<char *>(base);
    size_t o = 0;
    w.off = reinterpret_cast<int32_t *>(p);
    o += align256(sizeof(int32_t) * ((size_t)B + 1));
    w.img = reinterpret_cast<uint8_t *>(p + o);
    w.img_stride = (int64_t)align256(s.img_bytes);
    o += (size_t)B * w.img_stride;
    w.states = p + o;
    o += scaled_states_bytes((int64_t)B + ctas, s.H, d_h, s.r);
    w.bytes = o;
    return w;
}

bool fits(const ScaledPools &c, Shape &s) {
    if (c.d_h != 128 || c.G != 1 || !make_shape(c.H, c.r, s)) return false;
    if ((int64_t)c.num_pages * c.page_size + kTile >= INT32_MAX) return false;
    for (s.stages = kMaxStages; s.stages >= 6; --s.stages)
        if (Offsets(s).bytes <= kSmemMost) return tc_encode() != nullptr;
    return false;
}

}  // namespace

bool scaled_tc_covers(const ScaledPools &c) {
    Shape s;
    return fits(c, s);
}

size_t scaled_tc_ws_bytes(const ScaledPools &c, int B) {
    Shape s;
    if (!fits(c, s)) return 0;
    return layout(nullptr, s, B, device_sm_count(), c.d_h).bytes;
}

cudaError_t launch_decode_scaled_tc(const ScaledDecodeArgs &d, void *ws) {
    Shape s;
    const ScaledPools &c = d.c;
    if (!fits(c, s)) return cudaErrorInvalidValue;
    Args a;
    a.box_rows = c.page_size % 64 == 0 ? 64 : c.page_size % 32 == 0 ? 32 : 16;
    Maps maps;
    const int64_t rows = (int64_t)c.num_pages * c.page_size;
    if (!map_codes(&maps.k[0], c.code[0], rows, 128, a.box_rows) || !map_codes(&maps.v[0], c.code[1], rows, 128, a.box_rows) ||
        !map_codes(&maps.k[1], c.code[2], rows, c.H * c.r, a.box_rows) ||
        !map_codes(&maps.v[1], c.code[3], rows, c.H * c.r, a.box_rows))
        return cudaErrorInvalidValue;
    // (one CTA per SM; fewer where the requests cannot have as many units)
    const int sm = device_sm_count();
    const int64_t most = (int64_t)d.B * ((d.max_seq_len + kUnit - 1) / kUnit);
    const int ctas = (int)std::max<int64_t>(1, std::min<int64_t>(sm, most));
    const Ws w = layout(ws, s, d.B, sm, c.d_h);
    const int max_len = d.max_pages * c.page_size;
    PrepArgs p;
    p.q = static_cast<const __nv_bfloat16 *>(d.q);
    p.B_K = static_cast<const __nv_bfloat16 *>(d.B_K);
    p.seq_lens = d.seq_lens;
    p.img = w.img;
    p.img_stride = w.img_stride;
    p.off = w.off;
    p.B = d.B;
    p.max_len = max_len;
    p.scale_log2 = 1.4426950408889634f / sqrtf(128.f);
    cudaError_t e = launch_pdl(scaled_prep_kernel, dim3((unsigned)d.B + 1, c.H), dim3(128), 0, d.stream, p, s);
    if (e != cudaSuccess) return e;
    a.c = c;
    a.seq_lens = d.seq_lens;
    a.page_table = d.page_table;
    a.img = w.img;
    a.img_stride = w.img_stride;
    a.st = scaled_states(w.states, (int64_t)d.B + sm, c.H);
    a.status = d.status;
    a.B = d.B;
    a.max_pages = d.max_pages;
    a.max_len = max_len;
    const int bytes = Offsets(s).bytes;
    if (c.H <= 16) {
        if ((e = smem_limit_once(decode_scaled_kernel<16>, kSmemMost)) != cudaSuccess) return e;
        e = launch_pdl(decode_scaled_kernel<16>, dim3(ctas), dim3(kThreads), bytes, d.stream, maps, a, s);
    } else {
        if ((e = smem_limit_once(decode_scaled_kernel<32>, kSmemMost)) != cudaSuccess) return e;
        e = launch_pdl(decode_scaled_kernel<32>, dim3(ctas), dim3(kThreads), bytes, d.stream, maps, a, s);
    }
    if (e != cudaSuccess) return e;
    ScaledMergeArgs m;
    m.st = a.st;
    m.off = w.off;
    m.splits = 0;
    m.grid = ctas;
    m.seq_lens = d.seq_lens;
    m.max_len = max_len;
    m.leave = false;
    m.B_V = d.B_V;
    m.out = d.out;
    m.B = d.B;
    m.H = c.H;
    m.d_h = c.d_h;
    m.r = c.r;
    m.status = d.status;
    return launch_scaled_merge(m, d.stream);
}

}  // namespace lrkv
