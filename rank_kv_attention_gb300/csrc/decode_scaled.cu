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
// Scales: a token's exponent enters its score, d + e with d = x less the largest x so far,
// before the exponential: the value products take 2^(d + eS - MS) and 2^(d + eR - MR), each
// relative to the tile's largest per head, so tokens of loud and quiet blocks keep their
// precision next to each other.  The accumulators over tiles are relative to the largest d + eS
// and d + eR so far, not to the largest x: values lie between 2^-126 and 2^128, and neither a
// sum of loud ones nor a weight of a quiet one would fit in fp32 beside the value's own scale.
// Sums, maxima and the accumulators are fp32 in registers.
//
// Work: the requests' rows in units of 64 tokens, laid end to end and cut evenly
// over one CTA per SM; a CTA walks its tiles (two units of one request, or one).
// Each piece of a request in a CTA leaves a state in the workspace, and a second
// kernel merges and expands them by B_V[h].  A first, small kernel makes the q and p
// operands, each CTA's start and the places of each request's states.
//
// 24 warps: 0-15 scores and weights (thread = token = tensor-memory lane, a quarter of
// the heads each), 16-19 value accumulators (thread = column), one copies cache tiles,
// one issues the MMAs, one copies operands.  Order of the stream: keys of tile i + 1, then values of tile i, so a
// tile's softmax runs while the next keys arrive.
//
// Bound by HBM where rows are many, by a fixed 16 us (three launches in a row, the first
// tile's way through copy, scores, weights and values, merge 4 to 5) where they are few.  In a
// graph, H = 16, r = 48: 1 request of 1500 rows 16.3 us, 16 of 4096 rows 35.0 (3.4 TB/s, 17.4 at
// the copy bandwidth); r = 56, 64 ragged requests of 256 to 8192 rows 106 (5.2 TB/s; 82); H =
// 32, r = 32, 4 of 32768 rows 66 (4.6; 44.7).  The same requests took 27, 285, 1100 and 1052 in the
// form for any shape.  A tile's softmax is 5000 cycles of 16 heads and 7500 of 32, its values
// 4000 to 6000, next to 5700 to 8000 for its copies.
//
// Cache tiles are read once and leave L2 first: 16 requests of 4096 rows 36.5 us, 38.1 without
// (with two value accumulators in turn, where tensor memory has room, which frees the tensor
// core from the one that is being read: 4 of 32768 rows 73 us, 77 without both).
#include <algorithm>

#include "scaled_kernels.cuh"
#include "tc_common.cuh"

namespace lrkv {

namespace {

constexpr int kUnit = 64, kTile = 128;
constexpr int kStageBytes = kTile * 128;
// Scales of 16 tokens, which lie in one block: 2^eS_K (NaN: on no page), eS_V, then
// 2^eR_K and eR_V of every head.
constexpr int kScaleRow = 2 + 2 * 32 + 2;
constexpr int kMaxBoxes = 16, kMaxStages = 12;
// Warps: 16 of the softmax, 4 accumulating, then copies, operands, MMAs and tensor memory.
constexpr int kSoftmax = 512, kThreads = kSoftmax + 256;
constexpr int kWarpCopy = kSoftmax / 32 + 4, kWarpMma = kWarpCopy + 1, kWarpImage = kWarpCopy + 2, kWarpSpare = kWarpCopy + 3;
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
    uint16_t vbufs, vcols;     // value accumulators (tiles in turn), columns of one
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
    s.vcols = (uint16_t)(col - s.v0);
    s.vbufs = col + s.vcols <= 512 ? 2 : 1;
    col += (s.vbufs - 1) * s.vcols;
    s.tmem_cols = 32;
    while (s.tmem_cols < col) s.tmem_cols *= 2;
    s.img_bytes = (s.qrows + s.prows) * 128 + 8 * H;
    s.wrows = 2 * H;  // (a box's window may reach past the last head)
    for (int t = 0; t < s.boxes; ++t) s.wrows = std::max(s.wrows, 2 * s.ha[t] + s.nv[t]);
    s.wrows = std::max(s.wrows, (int)s.nv0 + 7) / 8 * 8;
    return true;
}

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t img_full[2], img_empty[2];
    uint64_t w_full[4], pv_done[2], v_empty[2];
    uint64_t meet[4];  // of the 128 softmax threads of a quarter of the heads
    uint64_t sc_full, sc_empty;
    // of every box (0: the shared rows): operand's offset, accumulator's column,
    // instruction descriptor and (keys) contraction steps
    alignas(16) uint4 kbox[kMaxBoxes + 1], vbox[kMaxBoxes + 1];
    uint64_t e_full[2], tmem_ready;
    uint32_t tmem;
};

// Shared memory after the ring of stages.
struct Offsets {
    int img, weights, red, fac, tops, scales, ar, bars, bytes;
    __host__ __device__ explicit Offsets(const Shape &s) {
        img = s.stages * kStageBytes;
        const int one = (s.img_bytes + 1023) / 1024 * 1024;
        weights = img + 2 * one;
        red = weights + 4 * s.wrows * 128;  // [2][4 quarters of the heads][maxima 3, sum][8][4 warps]
        fac = red + 2 * 4 * 4 * 8 * 4 * 4;  // [4][4][32]: what the shared sums and this tile's are multiplied by; the private
        tops = fac + 4 * 4 * 32 * 4;        // [2][32]: largest x - m + eS and x - m + eR of the request so far
        scales = tops + 2 * 32 * 4;         // [2][8 groups of 16 tokens][kScaleRow]
        ar = scales + 2 * 8 * kScaleRow * 4;  // [box][128]: the private accumulators
        bars = ar + s.boxes * 512;
        bytes = bars + (int)sizeof(Bars) + 1024;
    }
};

struct Maps {
    CUtensorMap k[2], v[2];  // S_K, R_K; S_V, R_V: [rows][bytes], box 128 bytes x box_rows
};

struct Args {
    ScaledPools c;
    const int32_t *seq_lens, *page_table;
    const int4 *starts;  // request, its length, first row, units of every CTA
    const uint8_t *img;  // operand images [B][img_bytes rounded up to 256]
    int64_t img_stride;
    ScaledStates st;
    int32_t *status;
    int B, max_pages, max_len, box_rows;
};

__device__ __forceinline__ int units_of(int L, int max_len) {
    return L >= 1 && L <= max_len ? (L + kUnit - 1) / kUnit : 0;
}

template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, uint32_t (&v)[2]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(taddr));
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
// that bring a tile's sums to log2 units; one more block the places of the states.
// ---------------------------------------------------------------------------
struct PrepArgs {
    const __nv_bfloat16 *q, *B_K;
    const int32_t *seq_lens;
    uint8_t *img;
    int64_t img_stride;
    int2 *places;  // of request b's states: first slot and count
    int4 *starts;  // where the tensor-core kernel's CTAs begin
    int32_t *status;
    int B, max_len, grid;
    float scale_log2;
};

__global__ void __launch_bounds__(128) scaled_prep_kernel(const __grid_constant__ PrepArgs P,
                                                          const __grid_constant__ Shape S) {
    __shared__ float qs[128], ps[64], part[128 * 8];
    __shared__ float red[8];
    __shared__ int sums[4];
    __shared__ uint32_t upto[128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == (unsigned)P.B) {
        if (blockIdx.y) return;
        // units of 64 rows, threads hold consecutive requests
        const int per = (P.B + 127) / 128, b0 = min(P.B, tid * per), b1 = min(P.B, b0 + per);
        uint32_t n = 0;
        for (int b = b0; b < b1; ++b) n += units_of(P.seq_lens[b], P.max_len);
        uint32_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) sums[warp] = (int)inc;
        __syncthreads();
        uint32_t U = 0, at = inc - n;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < warp) at += sums[w];
            U += sums[w];
        }
        upto[tid] = at + n;
        // CTA g takes the units [g U / G, (g + 1) U / G) (products below 2^32: at most 2^24
        // units); CTAs past the last unit have none, so that no request's CTAs have a gap
        const uint32_t G = min((uint32_t)P.grid, U);
        for (int b = b0; b < b1; ++b) {
            const uint32_t k = units_of(P.seq_lens[b], P.max_len);
            int2 place = make_int2(0, 0);
            if (k) {
                const uint32_t g0 = ((at + 1) * G - 1) / U, g1 = ((at + k) * G - 1) / U;
                place = make_int2(b + (int)g0, (int)(g1 - g0) + 1);
            } else {
                status_or(P.status, LRKV_STATUS_BAD_SEQLEN);
            }
            P.places[b] = place;
            at += k;
        }
        __syncthreads();
        for (int g = tid; g < P.grid; g += 128) {
            int4 start = make_int4(0, 0, 0, 0);  // request, its length, first row, units
            if (g < (int)G) {
                const uint32_t u0 = U * g / G, u1 = U * (g + 1) / G;
                int lo = 0, hi = 127;  // the thread whose requests hold unit u0
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if ((uint32_t)upto[mid] > u0) hi = mid;
                    else lo = mid + 1;
                }
                uint32_t from = lo ? upto[lo - 1] : 0;
                int b = lo * per, L;
                for (;; ++b) {
                    L = P.seq_lens[b];
                    const uint32_t k = units_of(L, P.max_len);
                    if (u0 < from + k) break;
                    from += k;
                }
                start = make_int4(b, L, (int)(u0 - from) * kUnit, (int)(u1 - u0));
            }
            P.starts[g] = start;
        }
        return;
    }
    const int b = blockIdx.x, h = blockIdx.y, r = S.r;
    const __nv_bfloat16 *B = P.B_K + (size_t)h * 128 * r;
    // p: groups of r / 8 threads take every `parts`-th channel, eight at most; all
    // loads are on their way together
    const int v8 = r / 8, parts = 128 / v8, pt = tid / v8, vc = tid % v8;
    uint4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (pt < parts && pt + i * parts < 128)
            w[i] = *reinterpret_cast<const uint4 *>(B + (size_t)(pt + i * parts) * r + 8 * vc);
    qs[tid] = __bfloat162float(P.q[((size_t)b * S.H + h) * 128 + tid]);
    __syncthreads();
    if (pt < parts) {
        float acc[8] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (pt + i * parts < 128) {
                const float q = qs[pt + i * parts];
                acc[0] = fmaf(q, bf16lo(w[i].x), acc[0]);
                acc[1] = fmaf(q, bf16hi(w[i].x), acc[1]);
                acc[2] = fmaf(q, bf16lo(w[i].y), acc[2]);
                acc[3] = fmaf(q, bf16hi(w[i].y), acc[3]);
                acc[4] = fmaf(q, bf16lo(w[i].z), acc[4]);
                acc[5] = fmaf(q, bf16hi(w[i].z), acc[5]);
                acc[6] = fmaf(q, bf16lo(w[i].w), acc[6]);
                acc[7] = fmaf(q, bf16hi(w[i].w), acc[7]);
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
    const int eq = bad ? 0 : needed_exp(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), 120);
    const int ep = bad ? 0 : needed_exp(fmaxf(fmaxf(red[4], red[5]), fmaxf(red[6], red[7])), 120);
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
    __device__ Walk() : b(0), L(0), tok(0), left(0), seg(0) {}
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

// HM: heads of the shape, rounded up to 16 or 32.
//
// Registers: 80 a thread at launch; the warps that copy and issue give 24 of theirs to
// the accumulating ones (16 * 32 * 80 + 4 * 32 * (104 + 56) = 768 * 80).
constexpr int kRegs = 80, kRegsFew = 56, kRegsMany = 104;
static_assert(kRegsFew + kRegsMany == 2 * kRegs, "what one group takes another has given");
template <int HM>
__global__ void __launch_bounds__(kThreads, 1)
    decode_scaled_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a,
                         const __grid_constant__ Shape S) {
    constexpr int HT = HM / 4;  // heads of a softmax thread
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const Offsets off(S);
    Bars &bar = *reinterpret_cast<Bars *>(smem + off.bars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = S.H, stages = S.stages, NB = S.boxes;
    const int img_stride = (S.img_bytes + 1023) / 1024 * 1024;

    // ---- set up while the kernels before this one end
    if (warp == kWarpImage) {  // (a lane initialises one to three barriers)
        if (lane < stages) {
            mbar_init(&bar.full[lane], 1);
            mbar_init(&bar.empty[lane], 1);
        } else if (lane >= 16 && lane < 18) {
            mbar_init(&bar.img_full[lane - 16], 1);
            mbar_init(&bar.img_empty[lane - 16], 1 + kSoftmax);
            mbar_init(&bar.e_full[lane - 16], 32);
        } else if (lane >= 18 && lane < 22) {
            mbar_init(&bar.w_full[lane - 18], kSoftmax);
            mbar_init(&bar.meet[lane - 18], 128);
        } else if (lane >= 22 && lane < 24) {
            mbar_init(&bar.pv_done[lane - 22], 1);
            mbar_init(&bar.v_empty[lane - 22], 128);
        } else if (lane == 24) {
            mbar_init(&bar.sc_full, 1);
            mbar_init(&bar.sc_empty, kSoftmax);
            mbar_init(&bar.tmem_ready, 1);
        }
        fence_barrier_init();
    } else if (warp == kWarpMma && lane <= NB) {
        const int x = lane;
        bar.kbox[x] = x ? make_uint4((S.qrows + S.prow[x - 1]) * 128, S.scol[x - 1], idesc_f8(S.n[x - 1], false),
                                     min(4, (H * S.r - 128 * (x - 1) + 31) / 32))
                        : make_uint4(0, 0, idesc_f8(S.qrows, false), 4);
        bar.vbox[x] = x ? make_uint4((S.wrows + 2 * S.ha[x - 1]) * 128, S.vcol[x - 1], idesc_f8(S.nv[x - 1], true), 0)
                        : make_uint4(0, S.v0, idesc_f8(S.nv0, true), 0);
    } else if (warp == kWarpCopy && elect_one()) {
        for (int k = 0; k < 2; ++k) {
            prefetch_tensormap(&maps.k[k]);
            prefetch_tensormap(&maps.v[k]);
        }
    }
    pdl_wait();  // (the operands' kernel is short: it is done by now)
    Walk w;
    {
        const int4 start = a.starts[blockIdx.x];
        w.b = start.x;
        w.L = start.y;
        w.tok = start.z;
        w.left = start.w;
    }
    __syncthreads();
    bool ok = true;

    if (warp >= kWarpCopy) {
        reg_dec<kRegsFew>();
        if (warp == kWarpCopy) {
            // ================= cache tiles =================
            // lane k looks up the pool row of the tile's k-th group of box_rows rows (past every
            // row, which reads as zeros, where its page is none)
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
            const uint64_t stream = l2_evict_first_policy();
            int s = 0, n = 0;  // stage, times the ring went round
            auto send = [&](const CUtensorMap *m, int rows, int row) {  // the keys or values of one tile
                const int groups = (rows + R - 1) / R;
                int y[8];
#pragma unroll
                for (int g = 0; g < 8; ++g) y[g] = __shfl_sync(0xffffffffu, row, g);
                for (int t = 0; t <= NB; ++t) {
                    if (n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bar.empty[s], (n - 1) & 1)) && ok;
                    if (!ok) return;
                    if (elect_one()) {
                        const CUtensorMap *map = m + (t > 0);
                        uint8_t *st = smem + s * kStageBytes;
                        const int x = t > 0 ? 128 * (t - 1) : 0;
                        mbar_arrive_expect_tx(&bar.full[s], groups * R * 128);
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            if (g < groups) tma_load_2d_hint(st + g * R * 128, map, x, y[g], &bar.full[s], stream);
                    }
                    __syncwarp();
                    if (++s == stages) {
                        s = 0;
                        ++n;
                    }
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
                for (int k = 0; k < stages; ++k)
                    if (k < s || n > 0) mbar_wait(&bar.full[k], (k < s ? n : n - 1) & 1);
        } else if (warp == kWarpImage) {
            // ================= operand images =================
            if (lane == 0) {
                pdl_launch_dependents();  // (the merge reads the places before its own wait)
                int last = -1;
                for (; ok && w.live(); w.next(a)) {
                    if (w.seg == last) continue;
                    const int s = last = w.seg, k = s & 1;
                    if (s >= 2 && !mbar_wait(&bar.img_empty[k], ((s >> 1) - 1) & 1)) {
                        ok = false;
                        --last;
                        break;
                    }
                    mbar_arrive_expect_tx(&bar.img_full[k], S.img_bytes);
                    bulk_load(smem + off.img + k * img_stride, a.img + w.b * a.img_stride, S.img_bytes, &bar.img_full[k]);
                }
                for (int s = max(0, last - 1); s <= last; ++s) mbar_wait(&bar.img_full[s & 1], (s >> 1) & 1);
            }
        } else if (warp == kWarpMma) {
            // ================= MMA issuer =================
            const uint32_t base = smem_u32(smem);
            ok = __all_sync(0xffffffffu, mbar_wait(&bar.tmem_ready, 0));
            const uint32_t tmem = bar.tmem;
            int s = 0, n = 0, i = 0;  // stage, times the ring went round; tile
            auto all_wait = [&](uint64_t *b, uint32_t parity) { return (bool)__all_sync(0xffffffffu, mbar_wait(b, parity)); };
            auto keys = [&](const Walk &t, bool first) -> bool {
                const uint32_t img = base + off.img + (t.seg & 1) * img_stride;
                if (first && !all_wait(&bar.img_full[t.seg & 1], (t.seg >> 1) & 1)) return false;
                if (i > 0 && !all_wait(&bar.sc_empty, (i - 1) & 1)) return false;
                const bool ends = t.ends();
                for (int x = 0; x <= NB; ++x) {
                    const uint4 box = bar.kbox[x];  // operand, accumulator, instruction, steps
                    if (!all_wait(&bar.full[s], n & 1)) return false;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t al = sw128_desc_lo(base + s * kStageBytes, 16), bl = sw128_desc_lo(img + box.x, 16);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < box.w) tc_mma_f8(tmem + box.y, al + 2 * k, bl + 2 * k, box.z, k != 0);
                        tc_commit(&bar.empty[s]);
                        if (x == NB) {
                            tc_commit(&bar.sc_full);
                            if (ends) tc_commit(&bar.img_empty[t.seg & 1]);
                        }
                    }
                    __syncwarp();
                    if (++s == stages) {
                        s = 0;
                        ++n;
                    }
                }
                return true;
            };
            auto values = [&](int rows, int j) -> bool {  // of the j-th tile
                if (!all_wait(&bar.w_full[j & 3], (j >> 2) & 1)) return false;
                const int vb = S.vbufs == 2 ? j & 1 : 0, round = S.vbufs == 2 ? j >> 1 : j;
                if (round > 0 && !all_wait(&bar.v_empty[vb], (round - 1) & 1)) return false;
                const int steps = (rows + 31) / 32;
                const uint32_t weights = base + off.weights + (j & 1) * 2 * S.wrows * 128;
                for (int x = 0; x <= NB; ++x) {
                    const uint4 box = bar.vbox[x];
                    if (!all_wait(&bar.full[s], n & 1)) return false;
                    tc_fence_after();
                    if (rows & 31) {
                        // rows past the end, of whatever bits, in the last group of 32: their
                        // weights are zero, and zero times a NaN is not
                        uint8_t *st = smem + s * kStageBytes;
                        for (int u = rows * 8 + lane; u < steps * 32 * 8; u += 32)
                            *reinterpret_cast<uint4 *>(st + u * 16) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (elect_one()) {
                        // 32 tokens an instruction: 32 rows of 128 bytes of A, 32 bytes of B's rows
                        const uint32_t al = sw128_desc_lo(base + s * kStageBytes, 16), bl = sw128_desc_lo(weights + box.x, 16);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < steps) tc_mma_f8(tmem + vb * S.vcols + box.y, al + 256 * k, bl + 2 * k, box.z, k != 0);
                        tc_commit(&bar.empty[s]);
                        if (x == NB) tc_commit(&bar.pv_done[j & 1]);
                    }
                    __syncwarp();
                    if (++s == stages) {
                        s = 0;
                        ++n;
                    }
                }
                return true;
            };
            if (ok && w.live()) {
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
        } else {
            // ================= tensor memory, scales of the tiles =================
            tmem_alloc(&bar.tmem, S.tmem_cols);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.tmem_ready);
            // lane: 16 tokens, a quarter of the heads
            const int grp = lane >> 2, quarter = lane & 3, hn = H / 4, h0 = quarter * hn;
            for (int i = 0; ok && w.live(); ++i, w.next(a)) {
                const int pos = w.tok + 16 * grp;
                int64_t eb = -1;
                if (16 * grp < w.rows()) {
                    const int32_t page = a.page_table[(size_t)w.b * a.max_pages + pos / a.c.page_size];
                    if (page >= 0 && page < a.c.num_pages)
                        eb = ((int64_t)page * a.c.page_size + pos % a.c.page_size) / a.c.block;
                }
                uint32_t sk = 0, sv = 0, k4[2] = {0, 0}, v4[2] = {0, 0};
                if (eb >= 0) {
                    const uint8_t *ek = a.c.exp[2] + eb * H + h0, *ev = a.c.exp[3] + eb * H + h0;
                    sk = a.c.exp[0][eb];
                    sv = a.c.exp[1][eb];
                    if (hn % 4 == 0) {  // (then these are aligned words)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (4 * j < hn) {
                                k4[j] = reinterpret_cast<const uint32_t *>(ek)[j];
                                v4[j] = reinterpret_cast<const uint32_t *>(ev)[j];
                            }
                    } else {
#pragma unroll 1
                        for (int j = hn - 1; j >= 0; --j) {
                            k4[1] = k4[1] << 8 | k4[0] >> 24;
                            v4[1] = v4[1] << 8 | v4[0] >> 24;
                            k4[0] = k4[0] << 8 | ek[j];
                            v4[0] = v4[0] << 8 | ev[j];
                        }
                    }
                }
                // the tile before the last is done with this buffer
                if (i > 1) ok = __all_sync(0xffffffffu, mbar_wait(&bar.w_full[(i - 2) & 3], ((i - 2) >> 2) & 1));
                if (!ok) break;
                float *row = reinterpret_cast<float *>(smem + off.scales) + ((i & 1) * 8 + grp) * kScaleRow;
                if (quarter == 0) {
                    row[0] = eb >= 0 ? exp2i(clamp_exp(sk)) : __uint_as_float(0x7fffffffu);
                    row[1] = (float)clamp_exp(sv);
                }
#pragma unroll 1
                for (int j = 0; j < hn; ++j) {
                    row[2 + h0 + j] = exp2i(clamp_exp((j < 4 ? k4[0] : k4[1]) >> (8 * (j & 3)) & 0xff));
                    row[34 + h0 + j] = (float)clamp_exp((j < 4 ? v4[0] : v4[1]) >> (8 * (j & 3)) & 0xff);
                }
                mbar_arrive(&bar.e_full[i & 1]);
            }
            if (!ok && lane == 0) status_or(a.status, LRKV_STATUS_TIMEOUT);
        }
    } else if (warp < kSoftmax / 32) {
        // ================= scores and weights =================
        // warp: tokens 32 (warp & 3) + lane of a tile, heads h0 .. h0 + hn - 1 (a quarter)
        const int hn = H / 4, grp = warp >> 2, h0 = grp * hn, token = 32 * (warp & 3) + lane;
        float l[HT], m = -INFINITY;  // m: of lane k's head h0 + k, the same in all four warps
        // (largest x - m + eS and x - m + eR: written and read by lane k of the first warp)
        float *tops = reinterpret_cast<float *>(smem + off.tops) + h0 + lane;
        uint32_t met = 0;
        auto meet = [&]() -> bool {  // the four warps of these heads
            mbar_arrive(&bar.meet[grp]);
            return __all_sync(0xffffffffu, mbar_wait(&bar.meet[grp], met++ & 1));
        };
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.tmem_ready, 0));
        const uint32_t lanes = bar.tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        int last = -1;
        for (int i = 0; ok && w.live(); ++i, w.next(a)) {
            const bool first = w.seg != last, ends = w.ends();
            const int seg = last = w.seg;
            if (first) {
                m = -INFINITY;
                if ((warp & 3) == 0 && lane < hn) tops[0] = tops[32] = -INFINITY;
#pragma unroll
                for (int k = 0; k < HT; ++k) l[k] = 0.f;
                ok = __all_sync(0xffffffffu, mbar_wait(&bar.img_full[seg & 1], (seg >> 1) & 1));
                if (!ok) break;
            }
            const float *f = reinterpret_cast<const float *>(smem + off.img + (seg & 1) * img_stride +
                                                             (S.qrows + S.prows) * 128) + h0;
            const float *scale = reinterpret_cast<const float *>(smem + off.scales) + ((i & 1) * 8 + token / 16) * kScaleRow;
            ok = __all_sync(0xffffffffu, mbar_wait(&bar.e_full[i & 1], (i >> 1) & 1) && mbar_wait(&bar.sc_full, i & 1));
            if (!ok) break;
            tc_fence_after();
            float x[HT];
            const float sk = scale[0];
            const bool there = token < w.rows() && sk == sk;
#pragma unroll
            for (int k = 0; k < HT; k += 2) {  // two heads' columns on their way together
                uint32_t vs[2][4], va[2][4], vb[2][4];
                bool two[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int h = h0 + min(k + j, hn - 1), ta = h * S.r / 128, tb = (h * S.r + S.r - 1) / 128;
                    two[j] = tb != ta;
                    tmem_ld4(lanes + 4 * h, vs[j]);
                    tmem_ld4(lanes + S.scol[ta] + 4 * (h - S.h0[ta]), va[j]);
                    if (two[j]) tmem_ld4(lanes + S.scol[tb], vb[j]);  // (the first head of that box)
                }
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    auto sum = [](const uint32_t (&v)[4]) {
                        return __uint_as_float(v[0]) + (__uint_as_float(v[1]) * 0.0625f + __uint_as_float(v[2]) * 0.001953125f);
                    };
                    float t = sum(va[j]);
                    if (two[j]) t += sum(vb[j]);
                    const int q = min(k + j, hn - 1);
                    x[k + j] = there ? sum(vs[j]) * (f[q] * sk) + t * (f[H + q] * scale[2 + h0 + q]) : -INFINITY;
                }
            }
            tc_fence_before();
            mbar_arrive(&bar.sc_empty);
            if (ends) mbar_arrive(&bar.img_empty[seg & 1]);  // (the factors were read)
            // (two buffers in turn: a warp writes the one after next only when all have met again)
            float *red = reinterpret_cast<float *>(smem + off.red) + ((i & 1) * 4 + grp) * HT * 16;
            const float es = scale[1];
            float er[HT];
            float mine[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < HT; ++k)
                if (k < hn) {
                    er[k] = there ? scale[34 + h0 + k] : 0.f;
                    const float m0 = warp_max(x[k]), d = x[k] - ref_of(m0), m1 = warp_max(d + es), m2 = warp_max(d + er[k]);
                    if (lane == k) {
                        mine[0] = m0;
                        mine[1] = m1;
                        mine[2] = m2;
                    }
                }
            if (lane < hn)
#pragma unroll
                for (int k = 0; k < 3; ++k) red[(k * HT + lane) * 4 + (warp & 3)] = mine[k];
            ok = meet();
            // the operand of the tile before the last has been read
            if (ok && i > 1) ok = __all_sync(0xffffffffu, mbar_wait(&bar.pv_done[i & 1], ((i >> 1) - 1) & 1));
            if (!ok) break;
            // lane k: what head h0 + k needs.  Of the weights' sum, weights relative to the running
            // maximum; of the operands, weights times scales relative to the tile's largest, which
            // becomes 2^8, and the value sums are relative to their own running maxima
            float alpha = 0.f, ref = 0.f, ms = 0.f, mr = 0.f;
            if (lane < hn) {
                const float4 v = *reinterpret_cast<const float4 *>(&red[lane * 4]);
                const float mn = fmaxf(fmaxf(m, fmaxf(v.x, v.y)), fmaxf(v.z, v.w));
                ref = ref_of(mn);
                float M[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {  // the warps' maxima are relative to their own largest scores
                    const float4 u = *reinterpret_cast<const float4 *>(&red[((1 + j) * HT + lane) * 4]);
                    M[j] = fmaxf(fmaxf(u.x + (v.x - ref), u.y + (v.y - ref)), fmaxf(u.z + (v.z - ref), u.w + (v.w - ref)));
                }
                ms = ref_of(M[0]) - 8.f;
                mr = ref_of(M[1]) - 8.f;
                const float down = m - ref;  // (-infinity: no row yet)
                alpha = ex2f(down);
                m = mn;
                if ((warp & 3) == 0) {
                    float *fac = reinterpret_cast<float *>(smem + off.fac) + (i & 3) * 4 * 32 + h0 + lane;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float was = tops[32 * j] + down, now = fmaxf(was, M[j]);
                        fac[64 * j] = ex2f(was - ref_of(now));
                        fac[64 * j + 32] = ex2f(M[j] - 8.f - ref_of(now));
                        tops[32 * j] = now;
                    }
                }
            }
            uint8_t *ws = smem + off.weights + (i & 1) * 2 * S.wrows * 128, *wr = ws + S.wrows * 128;
#pragma unroll
            for (int k = 0; k < HT; ++k)
                if (k < hn) {
                    const int h = h0 + k;
                    const float d = x[k] - __shfl_sync(0xffffffffu, ref, k), w = ex2f(d);
                    l[k] = l[k] * __shfl_sync(0xffffffffu, alpha, k) + w;
                    // both operands' terms, a pair at a time
                    const float y = ex2f(d + es - __shfl_sync(0xffffffffu, ms, k));
                    const float z = ex2f(d + er[k] - __shfl_sync(0xffffffffu, mr, k));
                    const uint16_t t1 = e4m3x2_from_f32(y, z);
                    const uint32_t h2 = f16x2_from_e4m3x2(t1);
                    const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
                    const uint16_t t2 = e4m3x2_from_f32((y - g.x) * 16.f, (z - g.y) * 16.f);
                    const uint32_t o1 = op_byte(2 * h, token), o2 = op_byte(2 * h + 1, token);
                    ws[o1] = (uint8_t)t1;
                    wr[o1] = (uint8_t)(t1 >> 8);
                    ws[o2] = (uint8_t)t2;
                    wr[o2] = (uint8_t)(t2 >> 8);
                }
            fence_proxy_async_smem();
            mbar_arrive(&bar.w_full[i & 3]);
            if (ends) {
                // the sums of all tokens: over the warp, then over the four warps
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < HT; ++k)
                    if (k < hn) {
                        float v = l[k];
#pragma unroll
                        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                        if (lane == k) sum = v;
                    }
                if (lane < hn) red[(3 * HT + lane) * 4 + (warp & 3)] = sum;
                if (!(ok = meet())) break;
                if ((warp & 3) == 0 && lane < hn) {
                    const float4 v = *reinterpret_cast<const float4 *>(&red[(3 * HT + lane) * 4]);
                    a.st.head[((int64_t)w.b + blockIdx.x) * H + h0 + lane] = make_float4(m, (v.x + v.y) + (v.z + v.w), tops[0], tops[32]);
                }
            }
        }
        if (!ok && lane == 0) status_or(a.status, LRKV_STATUS_TIMEOUT);
    } else {
        // ================= value accumulators: thread = column =================
        reg_inc<kRegsMany>();
        const int col = tid - kSoftmax, quad = warp & 3;
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.tmem_ready, 0));
        const uint32_t lanes = bar.tmem + ((uint32_t)(32 * quad) << 16);
        const uint32_t magic = 0xffffffffu / (uint32_t)S.r + 1u;  // 2^32 / r rounded up
        auto head_of = [&](int c) { return min((int)__umulhi((uint32_t)c, magic), H - 1); };
        float as[HM];
        float *ar = reinterpret_cast<float *>(smem + off.ar) + col;
        int last = -1, i = 0;
        for (; ok && w.live(); ++i, w.next(a)) {
            const bool first = w.seg != last;
            last = w.seg;
            if (first) {
#pragma unroll
                for (int h = 0; h < HM; ++h) as[h] = 0.f;
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&bar.w_full[i & 3], (i >> 2) & 1) &&
                                             mbar_wait(&bar.pv_done[i & 1], (i >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            const int vb = S.vbufs == 2 ? i & 1 : 0;
            const uint32_t from = lanes + vb * S.vcols;
            const float *fac = reinterpret_cast<const float *>(smem + off.fac) + (i & 3) * 4 * 32;
#pragma unroll
            for (int g = 0; g < HM / 16; ++g)
                if (16 * g < H) {
                    uint32_t v[32];
                    tmem_ld32(from + S.v0 + 32 * g, v);
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 al = *reinterpret_cast<const float4 *>(&fac[16 * g + k]);
                        const float4 fs = *reinterpret_cast<const float4 *>(&fac[32 + 16 * g + k]);
                        auto add = [&](int j, float x, float y) {
                            as[16 * g + k + j] = as[16 * g + k + j] * x +
                                                 (__uint_as_float(v[2 * (k + j)]) + __uint_as_float(v[2 * (k + j) + 1]) * 0.0625f) * y;
                        };
                        add(0, al.x, fs.x);
                        add(1, al.y, fs.y);
                        add(2, al.z, fs.z);
                        add(3, al.w, fs.w);
                    }
                }
            // a warp's 32 columns of a box belong to few heads (one or two from r = 32 on):
            // those heads' columns of D, four boxes on their way together
#pragma unroll 1
            for (int t0 = 0; t0 < NB; t0 += 4) {
                uint32_t v[4][2], u[4][2];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (t0 + j < NB) {
                        const int t = t0 + j, ha = S.ha[t], hA = head_of(128 * t + 32 * quad), hB = head_of(128 * t + 32 * quad + 31);
                        tmem_ld2(from + S.vcol[t] + 2 * (hA - ha), v[j]);
                        tmem_ld2(from + S.vcol[t] + 2 * (hB - ha), u[j]);
                    }
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (t0 + j < NB) {
                        const int t = t0 + j, ha = S.ha[t], hA = head_of(128 * t + 32 * quad), hB = head_of(128 * t + 32 * quad + 31);
                        const int h = head_of(128 * t + col);
                        for (int k = hA + 1; k < hB; ++k) {
                            uint32_t x[2];
                            tmem_ld2(from + S.vcol[t] + 2 * (k - ha), x);
                            tmem_wait_ld();
                            if (h == k) {
                                v[j][0] = x[0];
                                v[j][1] = x[1];
                            }
                        }
                        const bool up = h == hB;
                        const float y = __uint_as_float(up ? u[j][0] : v[j][0]) + __uint_as_float(up ? u[j][1] : v[j][1]) * 0.0625f;
                        ar[128 * t] = first ? y * fac[96 + h] : ar[128 * t] * fac[64 + h] + y * fac[96 + h];
                    }
            }
            tc_fence_before();
            mbar_arrive(&bar.v_empty[vb]);
            if (w.ends()) {
                float *acc = a.st.acc + ((int64_t)w.b + blockIdx.x) * H * (128 + S.r);
#pragma unroll
                for (int h = 0; h < HM; ++h)
                    if (h < H) acc[h * 128 + col] = as[h];
                for (int t = 0; t < NB; ++t)
                    if (128 * t + col < H * S.r) acc[H * 128 + 128 * t + col] = ar[128 * t];
            }
        }
        if (!ok && lane == 0) status_or(a.status, LRKV_STATUS_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpSpare) {
        tc_fence_after();
        tmem_dealloc(bar.tmem, S.tmem_cols);
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

template <typename K>
int launch_registers(K *kernel) {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, kernel) == cudaSuccess ? f.numRegs : 0;
}

// Workspace: places of the states, operand images, states of up to B + CTAs pieces.
struct Ws {
    int2 *places;
    int4 *starts;
    uint8_t *img;
    int64_t img_stride;
    void *states;
    size_t bytes;
};
Ws layout(void *base, const Shape &s, int B, int ctas, int d_h) {
    Ws w;
    char *p = static_cast<char *>(base);
    size_t o = 0;
    w.places = reinterpret_cast<int2 *>(p);
    o += align256(sizeof(int2) * (size_t)B);
    w.starts = reinterpret_cast<int4 *>(p + o);
    o += align256(sizeof(int4) * (size_t)ctas);
    w.img = reinterpret_cast<uint8_t *>(p + o);
    w.img_stride = (int64_t)align256(s.img_bytes);
    o += (size_t)B * w.img_stride;
    w.states = p + o;
    o += scaled_states_bytes((int64_t)B + ctas, s.H, d_h, s.r);
    w.bytes = o;
    return w;
}

// Whether the compiler gave the kernels the registers that their warps hand on: taking more than
// the launch has would wait forever.
bool registers_fit() {
    static const bool fit = launch_registers(decode_scaled_kernel<16>) == kRegs &&
                            launch_registers(decode_scaled_kernel<32>) == kRegs;
    return fit;
}

bool fits(const ScaledPools &c, Shape &s) {
    if (c.d_h != 128 || c.G != 1 || !make_shape(c.H, c.r, s)) return false;
    if ((int64_t)c.num_pages * c.page_size + kTile >= INT32_MAX) return false;
    for (s.stages = kMaxStages; s.stages >= 6; --s.stages)
        if (Offsets(s).bytes <= kSmemMost) return tc_encode() != nullptr && registers_fit();
    return false;
}

}  // namespace

bool scaled_tc_covers(const ScaledPools &c) {
    Shape s;
    return fits(c, s);
}

// CTAs of a call: one per SM; fewer where the requests cannot have as many units.
static int ctas_of(int B, int max_seq_len) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), B * (((int64_t)max_seq_len + kUnit - 1) / kUnit)));
}

size_t scaled_tc_ws_bytes(const ScaledPools &c, int B, int max_seq_len) {
    Shape s;
    if (!fits(c, s)) return 0;
    return layout(nullptr, s, B, ctas_of(B, max_seq_len), c.d_h).bytes;
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
    const int ctas = ctas_of(d.B, d.max_seq_len);
    const auto kernel = c.H <= 16 ? decode_scaled_kernel<16> : decode_scaled_kernel<32>;
    const Ws w = layout(ws, s, d.B, ctas, c.d_h);
    const int max_len = d.max_pages * c.page_size;
    PrepArgs p;
    p.q = static_cast<const __nv_bfloat16 *>(d.q);
    p.B_K = static_cast<const __nv_bfloat16 *>(d.B_K);
    p.seq_lens = d.seq_lens;
    p.img = w.img;
    p.img_stride = w.img_stride;
    p.places = w.places;
    p.starts = w.starts;
    p.status = d.status;
    p.grid = ctas;
    p.B = d.B;
    p.max_len = max_len;
    p.scale_log2 = 1.4426950408889634f / sqrtf(128.f);
    cudaError_t e = launch_pdl(scaled_prep_kernel, dim3((unsigned)d.B + 1, c.H), dim3(128), 0, d.stream, p, s);
    if (e != cudaSuccess) return e;
    a.c = c;
    a.seq_lens = d.seq_lens;
    a.page_table = d.page_table;
    a.starts = w.starts;
    a.img = w.img;
    a.img_stride = w.img_stride;
    a.st = scaled_states(w.states, (int64_t)d.B + ctas, c.H);
    a.status = d.status;
    a.B = d.B;
    a.max_pages = d.max_pages;
    a.max_len = max_len;
    const int bytes = Offsets(s).bytes;
    if ((e = smem_limit_once(kernel, kSmemMost)) != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(ctas), dim3(kThreads), bytes, d.stream, maps, a, s);
    if (e != cudaSuccess) return e;
    ScaledMergeArgs m;
    m.st = a.st;
    m.places = w.places;
    m.splits = 0;
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
