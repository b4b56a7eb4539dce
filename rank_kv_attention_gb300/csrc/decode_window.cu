// Decode through a sliding window with sinks, on tensor cores (bf16 and 8-bit
// caches, d_h = 128; the shapes of decode_tile.cuh).
//
// Request b's query sees its last `window` rows and its first `sinks` rows.
// Those two runs of rows, each widened to whole 16-row tiles, are laid end to
// end as the request's `virtual rows` (VirtualRows); a tile of virtual rows is
// a tile of cache rows, and rows of a tile that the query does not see are
// masked.  So work is proportional to the window, whatever the history's
// length, and a page without a visible row is never touched.
//
// One thread-block cluster works on one run of virtual rows at a time (a
// `segment` of one request); its CTAs take equal shares of the tiles.
//   * A warp of its own brings a CTA's tiles by TMA into a ring of slots, each the
//     key half (S_K and all heads' R_K) or the value half of a tile, so a key half
//     makes room as soon as its scores exist.
//   * A warp takes four heads and one tile at a time (see HeadState): eight warps
//     cover 32 heads, or twice 16, and then two groups of four warps take the
//     even and the odd tiles.
//   * The private queries p = q B_K[h] are formed by the cluster while its first
//     tiles are on the way, each CTA for its H / CL heads, and sent to every CTA.
//   * At the end of a segment each CTA sends its state (m, l, accS, accR) of head
//     h to the CTA of the cluster that owns the head (distributed shared memory);
//     the owner merges the states by the log-sum-exp rule and expands by B_V[h].
// Nothing waits for another cluster and there are no atomics on global memory:
// two calls can share the GPU in any order, and results repeat bit for bit.
// While a cluster merges one segment, its ring already fetches the next one's
// tiles.
//
// A segment is a whole request, and cluster c takes requests c, c + NC, ...: the
// kernel is the whole decode, in one launch.  Only for few requests with long
// windows, which whole requests would put on few SMs, a request is split over S
// clusters whose states a combine kernel merges.
//
// In a graph, 16 heads, r = 48, bf16 unless noted: 1 request, window 512, 11.1 us
// and 16 requests, window 1024, 22 us (59 MB): latency, of which 8 to 9 us are a
// launch's and a segment's fixed cost and 0.67 us a tile (57 KB) per CTA; 64 ragged
// requests, window 4000, r = 56: 132 us, 6.2 TB/s, 92% of the measured copy bandwidth,
// DRAM reads 1.004 of the visible rows; 32 requests, window 2048, 8-bit: 46 us, where
// the conversions of codes bound a tile (1.0 us for 28 KB); 4 requests of 32 heads,
// r = 32, window 8192, split: 34 us, 4.5 TB/s.
#include <algorithm>
#include <mutex>

#include "decode_tile.cuh"
#include "tc_pair.cuh"

namespace lrkv {

namespace {

constexpr int kTS = 16;          // rows per tile
constexpr int kMaxSplits = 32;   // clusters per request at most (a warp of the combine weighs them)
constexpr int kBars = 16;        // half turns that can be on the way: more than there are slots

template <int H_, int R_, bool Q8_, int NGRP_>
struct WinCfg {
    static constexpr int H = H_, R = R_, NGRP = NGRP_, DH = 128, W = DH + R;
    static constexpr bool Q8 = Q8_;
    static constexpr int EB = Q8 ? 1 : 2;        // bytes per cache element
    static constexpr int NCW = 8, NT = NCW * 32;  // warps (threads) that own heads
    // and a warpgroup whose first warp copies: registers are handed over between
    // whole warpgroups.  A block of 384 threads has 168 registers each; 56 for
    // the copying group leave 224 for the others (128 x 56 + 256 x 224 = 384 x 168)
    static constexpr int THREADS = NT + 128, REG_COPY = 56, REG_HEADS = 224;
    static_assert(128 * REG_COPY + NT * REG_HEADS <= THREADS * 168, "registers of the block");
    static constexpr int HPW = 4, NH = 2;        // heads per warp, head slots per thread
    static constexpr int HW = H / HPW;           // warps that cover the heads
    static constexpr int NG = NCW / HW;          // groups of such warps (tiles taken in turn)
    static constexpr int KSP = HPW * R / 16;     // k-steps (and m-tiles) of a warp's private columns
    // one slot: the shared rows, then all heads' private rows, in 16-row x 128-byte swizzled boxes
    static constexpr int S_BYTES = NGRP * DH * EB * kTS, R_BYTES = H * R * EB * kTS;
    static constexpr int SLOT = S_BYTES + R_BYTES;
    static constexpr int NKB = kTS * H * 2;      // joint key norms of a tile (bf16)
    static constexpr int WS = W + 4;             // a state: accS, accR, m, l, padding (16-byte rows)
    // everything but the ring and its norms
    static constexpr int FIXED = H * R * 4 + H * 4 + NG * H * WS * 4 + 32 * 4 + kBars * 8 * 2 + kBars * 4 + 64;
    // as many slots as fit, up to 12: more in flight than the latency needs
    // only delays the first tile
    static constexpr int FIT = (227 * 1024 - 1024 - FIXED) / (SLOT + NKB);
    static constexpr int SLOTS = FIT > 12 ? 12 : FIT;
    static constexpr int OFF_NK = SLOTS * SLOT;
    // private queries [H][R]: rounded values, then their remainders (bf16, or f16
    // for an 8-bit cache, scaled: [H] inverse scales)
    static constexpr int OFF_P = OFF_NK + SLOTS * NKB;
    static constexpr int OFF_PSC = OFF_P + H * R * 4;
    // states of the heads this CTA owns, from every group of warps of every CTA of
    // the cluster: [NG CL][H / CL][WS]
    static constexpr int OFF_RECV = OFF_PSC + H * 4;
    static constexpr int OFF_WTS = OFF_RECV + NG * H * WS * 4;  // weights of the states [H / CL][NG CL]
    // one full and one empty barrier per half turn (the key halves or the value
    // halves of the tiles that the groups take at once), kBars halves in turn
    static constexpr int OFF_BAR = OFF_WTS + 32 * 4;
    static constexpr int OFF_EMPTY = OFF_BAR + kBars * 8;
    static constexpr int OFF_CB = OFF_EMPTY + kBars * 8;     // cluster barriers
    static constexpr int OFF_OK = OFF_CB + 32;               // per half turn: bit i, tile i's page id is valid
    static constexpr int SMEM = OFF_OK + kBars * 4 + 1024;   // + alignment slack
    static_assert(H == 16 || H == 32, "four or eight warps cover the heads");
    static_assert((HPW * R) % 16 == 0 && (H * R * EB) % 128 == 0, "whole k-steps and boxes");
    static_assert(NGRP == 1 || (H / NGRP) % HPW == 0, "a warp's heads share one group");
    static_assert(SLOT % 1024 == 0 && NKB % 128 == 0, "swizzled boxes on 1 KB, norms on 128 bytes");
    static_assert(SLOTS >= 4 && SLOTS <= kBars - 2, "a turn's key and value halves; barriers for every slot");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct WinMaps {
    CUtensorMap sk, sv, rk, rv, nk;
};

struct WinParams {
    const __nv_bfloat16 *q, *B_K, *B_V;
    __nv_bfloat16 *out;
    const int32_t *seq_lens, *page_table, *req_row;
    int B, max_pages, num_pages, page_size, max_len, window, sinks;
    int splits, norm;  // clusters per request; the cache holds joint key norms
    float scale_log2;
    float4 sc;  // 8-bit cache: pool scales of S_K, S_V, R_K, R_V
    float *ml, *acc;   // states for the combine: [B splits][H][2], [B splits][H][128 + r]
    int32_t *status;
};

// A request's visible rows as tiles: virtual rows [0, A) are cache rows [0, A)
// (the sinks), virtual row v >= A is cache row v + shift (the window).
struct VirtualRows {
    int32_t sinks, first, A, shift, total;
    __device__ __forceinline__ VirtualRows(int32_t L, const WinParams &P) {
        const VisibleRows v(L, P.window, P.sinks);
        sinks = v.sinks;
        first = v.first;
        const int32_t w0 = v.first / kTS * kTS;
        A = (v.sinks + kTS - 1) / kTS * kTS;
        if (A >= w0) {  // the runs touch (or there are no sinks): one run
            A = 0;
            shift = v.sinks ? 0 : w0;
        } else {
            shift = w0 - A;
        }
        total = (L < 1 || L > P.max_len) ? 0 : L - shift;
    }
    __device__ __forceinline__ int32_t row(int32_t v) const { return v < A ? v : v + shift; }
};

// A segment: virtual rows [va, vb) of a request.
struct Segment {
    int b;
    int32_t L;       // the request's length
    int32_t va, vb;
    // the cluster's k-th (false past its last one)
    __device__ __forceinline__ bool at(const WinParams &P, int k, int cid, int NC) {
        const int64_t i = cid + (int64_t)k * NC;
        if (i >= (int64_t)P.B * P.splits) return false;
        b = (int)(i / P.splits);
        const int s = (int)(i - (int64_t)b * P.splits);
        L = P.seq_lens[b];
        const int32_t total = VirtualRows(L, P).total, n = (total + kTS - 1) / kTS;
        va = (int32_t)((int64_t)n * s / P.splits) * kTS;
        vb = min(total, (int32_t)((int64_t)n * (s + 1) / P.splits) * kTS);
        return true;
    }
};

// The CTA's whole tiles of a segment: virtual rows [t0, t1).
struct Range {
    int32_t t0, t1;
    __device__ __forceinline__ Range(const Segment &w, int rank, int CL) {
        const int32_t a = w.va / kTS, n = (w.vb + kTS - 1) / kTS - a;
        t0 = (a + n * rank / CL) * kTS;
        t1 = (a + n * (rank + 1) / CL) * kTS;
    }
};

// The warps that own heads (not the copying one) meet here.
__device__ __forceinline__ void heads_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// Arrive on an mbarrier of a CTA of the cluster, releasing this CTA's writes
// (after a __syncwarp or heads_sync, those of the warps that met there) to the
// cluster.
__device__ __forceinline__ void arrive_cluster(uint32_t cl_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cl_addr) : "memory");
}
// mbar_wait whose completion acquires the arriving CTAs' writes.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; "
            "selp.u32 %0, 1, 0, p; }"
            : "=r"(ok)
            : "r"(a), "r"(parity)
            : "memory");
        if (ok) return true;
        if (it == 0) t0 = globaltimer_ns();
        else if ((it & 255u) == 255u && globaltimer_ns() - t0 > 2000000000ull) return false;
    }
}
// Pairs of fp32 (PTX f32x2 arithmetic, sm_100 family).
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f32x2_unpack(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// 2^x of a softmax weight, x <= kLazyMax (PTX ex2.approx.ftz: ~2 ulp; weights
// below 2^-126 become 0).
__device__ __forceinline__ float exp2_weight(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Stores to shared memory of a CTA of the cluster.
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p, size_t bytes, int tid, int n) {
    for (size_t o = (size_t)tid * 128; o < bytes; o += (size_t)n * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p) + o));
}

// ---------------------------------------------------------------------------
// One warp's four heads over a segment.  Products run as mma.m16n8k16 with the
// 16 tile rows (scores) or 16 value columns (values) as M and the heads as N.  Of
// the eight N columns, column n < 4 is head n and column 4 + n the low half of
// head n's operand: p and the softmax weights enter as a rounded value and its
// remainder (bf16 or f16 pairs, ~16 or ~22 significant bits) in one instruction,
// and the two columns are added afterwards.  Two heads a warp and separate
// instructions for the halves (the full decode's form) take 48 products a tile
// for r = 48 on each of eight warps, this 40 on each of four.
// ---------------------------------------------------------------------------
template <class C>
struct HeadState {
    const int wq, grp, lane;       // this warp's heads are 4 wq .. 4 wq + 3; its group
    const int gq, tq;              // mma fragment coordinates
    const int hl, j;               // this lane's (head slot, tile row)
    const bool hi;                 // B fragment: column gq is a high half
    uint32_t oks, okr, ovs, ovr;   // fragment offsets in a slot, of the first k-step (m-tile)
    float accS[8][4], accR[C::KSP][4];
    float m[C::NH], l[C::NH];      // l: this lane's rows only
    uint32_t qb[8][2], pb[C::KSP][2];
    float fS[2], fR[2];  // 8-bit cache: score factors of columns 2tq, 2tq + 1

    __device__ __forceinline__ HeadState()
        : wq((int)(threadIdx.x >> 5) % C::HW), grp((int)(threadIdx.x >> 5) / C::HW), lane(threadIdx.x & 31),
          gq((threadIdx.x & 31) >> 2), tq(threadIdx.x & 3), hl((threadIdx.x & 31) >> 4), j(threadIdx.x & 15),
          hi(((threadIdx.x & 31) >> 2) < C::HPW) {
        fS[0] = fS[1] = fR[0] = fR[1] = 1.f;
        oks = ovs = okr = ovr = 0;
        if constexpr (!C::Q8) {
            const int mi = lane >> 3, rk = (mi & 1) * 8 + (lane & 7), rv = (mi >> 1) * 8 + (lane & 7);
            // first 16-byte chunk of the group of this warp's heads, and of its private columns
            const int sg = (wq * C::HPW) / (C::H / C::NGRP) * (C::DH / 8), cw = wq * (C::HPW * C::R / 8);
            oks = box_chunk_rows<kTS>(rk, sg + (mi >> 1));
            ovs = box_chunk_rows<kTS>(rv, sg + (mi & 1));
            okr = C::S_BYTES + box_chunk_rows<kTS>(rk, cw + (mi >> 1));
            ovr = C::S_BYTES + box_chunk_rows<kTS>(rv, cw + (mi & 1));
        }
    }
    __device__ __forceinline__ int head(int i) const { return wq * C::HPW + hl + 2 * i; }  // of slot i
    // slot offset two chunks k times after that of `o`, whose chunk is a
    // multiple of eight (or one more)
    __device__ __forceinline__ static uint32_t at_step(uint32_t o, int k) {
        return (o ^ ((2u * (k & 3)) << 4)) + (uint32_t)(k >> 2) * (kTS * 128);
    }
    // the same for the warp's private columns, which may start at chunk 4 of eight
    __device__ __forceinline__ uint32_t private_at(uint32_t o, int k) const {
        if constexpr ((C::HPW * C::R / 8) % 8 == 0) {
            return at_step(o, k);
        } else {
            const int carry = (((wq * (C::HPW * C::R / 8)) & 7) + 2 * (k & 3)) >> 3;  // past the eighth chunk
            return (o ^ ((2u * (k & 3)) << 4)) + (uint32_t)((k >> 2) + carry) * (kTS * 128);
        }
    }

    // Query fragments of request b (global loads) and an empty state.
    __device__ __forceinline__ void begin_shared(const WinParams &P, int b) {
#pragma unroll
        for (int i = 0; i < C::NH; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) accS[t][e] = 0.f;
#pragma unroll
        for (int t = 0; t < C::KSP; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) accR[t][e] = 0.f;
        const __nv_bfloat16 *qrow = P.q + ((size_t)b * C::H + wq * C::HPW + (gq & 3)) * C::DH;
        if constexpr (!C::Q8) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                qb[ks][0] = hi ? ld_u32(qrow + ks * 16 + 2 * tq) : 0u;
                qb[ks][1] = hi ? ld_u32(qrow + ks * 16 + 2 * tq + 8) : 0u;
            }
        } else {
            // 8-bit cache: the order of a k-step's 16 indices is free as long as
            // both operands use the same one: slot order 4 tq + e (one 32-bit
            // word of codes per row).  q enters as f16 after an exact power-of-two
            // scaling that brings the head's largest |value| into [2^14, 2^15)
            float qv[8][4], mq = 0.f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint2 u = *reinterpret_cast<const uint2 *>(qrow + ks * 16 + 4 * tq);
                qv[ks][0] = bf16lo(u.x); qv[ks][1] = bf16hi(u.x);
                qv[ks][2] = bf16lo(u.y); qv[ks][3] = bf16hi(u.y);
#pragma unroll
                for (int e = 0; e < 4; ++e) mq = fmaxf(mq, fabsf(qv[ks][e]));
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, o));
            const int eq = f16_range_shift(mq);
            const float uq = hi ? exp2i(eq) : 0.f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                qb[ks][0] = hi ? pack_f16(qv[ks][0] * uq, qv[ks][1] * uq) : 0u;
                qb[ks][1] = hi ? pack_f16(qv[ks][2] * uq, qv[ks][3] * uq) : 0u;
            }
            const float f = P.sc.x * exp2i(-eq);  // column n's factor sits in lanes 4n ..
            fS[0] = __shfl_sync(0xffffffffu, f, 8 * tq);
            fS[1] = __shfl_sync(0xffffffffu, f, 8 * tq + 4);
        }
    }
    // blockdiag(p)^T fragments: entry (k, n) is p[head n][k - n R] when k lies
    // in head n's columns of the warp, else 0; ph: this lane's halves of the
    // warp's heads' p (rounded values or remainders), R apart; sc: their scales.
    __device__ __forceinline__ void begin_private(const WinParams &P, const uint16_t *ph, const float *sc) {
        const int n = gq & 3;
#pragma unroll
        for (int ks = 0; ks < C::KSP; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = C::Q8 ? ks * 16 + 4 * tq + 2 * e : ks * 16 + 2 * tq + 8 * e;
                pb[ks][e] = k / C::R == n ? *reinterpret_cast<const uint32_t *>(ph + k) : 0u;
            }
        if constexpr (C::Q8) {  // factors of columns 2tq, 2tq + 1
            fR[0] = P.sc.z * sc[(2 * tq) & 3];
            fR[1] = P.sc.z * sc[(2 * tq + 1) & 3];
        }
    }

    // Scores of the key slot st, scaled (log2 units): lane (hl, j) gets row j of
    // heads head(0), head(1).  nk: the tile's key norms.
    __device__ __forceinline__ void scores(const WinParams &P, const uint8_t *st, const uint8_t *nk, bool valid,
                                           float (&s)[C::NH]) const {
        float cS[2][4], cR[2][4];  // two chains each
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) cS[k][e] = cR[k][e] = 0.f;
        if constexpr (C::Q8) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint32_t w0 = lds_u32(st + box_chunk_rows<kTS>(gq, ks) + 4 * tq);
                const uint32_t w1 = lds_u32(st + box_chunk_rows<kTS>(gq + 8, ks) + 4 * tq);
                const uint32_t a[4] = {f16x2_lo(w0), f16x2_lo(w1), f16x2_hi(w0), f16x2_hi(w1)};
                mma_f16_16816(cS[ks & 1], a, qb[ks][0], qb[ks][1]);
            }
            const int cw = wq * (C::HPW * C::R / 16);  // first 16-byte chunk of the warp's columns
            const uint8_t *r = st + C::S_BYTES + 4 * tq;
#pragma unroll
            for (int ks = 0; ks < C::KSP; ++ks) {
                const uint32_t w0 = lds_u32(r + box_chunk_rows<kTS>(gq, cw + ks));
                const uint32_t w1 = lds_u32(r + box_chunk_rows<kTS>(gq + 8, cw + ks));
                const uint32_t a[4] = {f16x2_lo(w0), f16x2_lo(w1), f16x2_hi(w0), f16x2_hi(w1)};
                mma_f16_16816(cR[ks & 1], a, pb[ks][0], pb[ks][1]);
            }
        } else {
            const uint32_t b = smem_u32(st);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                uint32_t a[4];
                ldmatrix_x4(b + at_step(oks, ks), a[0], a[1], a[2], a[3]);
                mma_bf16_16816(cS[ks & 1], a, qb[ks][0], qb[ks][1]);
            }
#pragma unroll
            for (int ks = 0; ks < C::KSP; ++ks) {
                uint32_t a[4];
                ldmatrix_x4(b + private_at(okr, ks), a[0], a[1], a[2], a[3]);
                mma_bf16_16816(cR[ks & 1], a, pb[ks][0], pb[ks][1]);
            }
        }
        float c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = cS[0][e] + cS[1][e], y = cR[0][e] + cR[1][e];
            c[e] = C::Q8 ? fS[e & 1] * x + fR[e & 1] * y : x + y;
            c[e] += __shfl_xor_sync(0xffffffffu, c[e], 2);  // columns n and 4 + n
        }
#pragma unroll
        for (int i = 0; i < C::NH; ++i) {
            // D[row j][head n = hl + 2i] sits in lane (j % 8) * 4 + i, register hl + 2 (j / 8)
            const int src = (j & 7) * 4 + i;
            const float v0 = __shfl_sync(0xffffffffu, c[0], src);
            const float v1 = __shfl_sync(0xffffffffu, c[1], src);
            const float v2 = __shfl_sync(0xffffffffu, c[2], src);
            const float v3 = __shfl_sync(0xffffffffu, c[3], src);
            float x = ((j < 8) ? (hl ? v1 : v0) : (hl ? v3 : v2)) * P.scale_log2;
            if (P.norm)  // joint key norm of (row j, head)
                x *= __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(nk)[j * C::H + head(i)]);
            s[i] = valid ? x : -INFINITY;
        }
    }

    // factors f[i] of the heads of each slot, as factors of columns 2tq, 2tq + 1
    // (heads (2tq + e) % 4: head n sits in slot n >> 1 of the half-warp n & 1)
    __device__ __forceinline__ void column_factors(const float (&f)[C::NH], float &a0, float &a1) const {
        const float x0 = __shfl_sync(0xffffffffu, f[0], 0), x1 = __shfl_sync(0xffffffffu, f[0], 16);
        const float y0 = __shfl_sync(0xffffffffu, f[1], 0), y1 = __shfl_sync(0xffffffffu, f[1], 16);
        a0 = (tq & 1) ? y0 : x0;
        a1 = (tq & 1) ? y1 : x1;
    }
    __device__ __forceinline__ void rescale(const float (&f)[C::NH]) {
        float a0, a1;
        column_factors(f, a0, a1);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            accS[t][0] *= a0; accS[t][1] *= a1; accS[t][2] *= a0; accS[t][3] *= a1;
        }
#pragma unroll
        for (int t = 0; t < C::KSP; ++t) {
            accR[t][0] *= a0; accR[t][1] *= a1; accR[t][2] *= a0; accR[t][3] *= a1;
        }
    }

    // Softmax weights of the scores (in s, replaced) against the running
    // maximum, which only moves when a row exceeds it by kLazyMax; then the
    // accumulators are rescaled.
    __device__ __forceinline__ void softmax(float (&s)[C::NH]) {
        if (__any_sync(0xffffffffu, s[0] > m[0] + kLazyMax || s[1] > m[1] + kLazyMax)) {
            float al[C::NH];
#pragma unroll
            for (int i = 0; i < C::NH; ++i) {
                float mx = s[i];
#pragma unroll
                for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float m_new = mx > m[i] + kLazyMax ? mx : m[i];
                al[i] = m_new == m[i] ? 1.f : exp2f(m[i] - m_new);
                m[i] = m_new;
                l[i] *= al[i];
            }
            rescale(al);
        }
#pragma unroll
        for (int i = 0; i < C::NH; ++i) {
            s[i] = s[i] == -INFINITY ? 0.f : exp2_weight(s[i] - m[i]);
            l[i] += s[i];
        }
    }

    // accS += S_V^T . P^T, accR += R_V^T(warp columns) . P^T over the value slot.
    // MASK: rows outside msk may hold anything.
    template <bool MASK>
    __device__ __forceinline__ void values(const uint8_t *st, const float (&e)[C::NH], uint32_t msk) {
        // column gq of the B fragment: head gq % 4's weights of rows 2tq, 2tq + 1,
        // 2tq + 8, 2tq + 9; each lane packs its weight's two halves
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < C::NH; ++i) {
            float h;
            uint32_t u;
            if constexpr (C::Q8) {
                h = __half2float(__float2half_rn(e[i]));
                u = pack_f16(h, e[i] - h);
            } else {
                h = __bfloat162float(__float2bfloat16_rn(e[i]));
                u = pack_bf16(h, e[i] - h);
            }
            const int sl = (gq & 1) * 16 + 2 * tq;
            const uint32_t y[4] = {__shfl_sync(0xffffffffu, u, sl), __shfl_sync(0xffffffffu, u, sl + 1),
                                   __shfl_sync(0xffffffffu, u, sl + 8), __shfl_sync(0xffffffffu, u, sl + 9)};
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = (i == 0 || (gq & 2)) ? y[q] : x[q];
        }
        const uint32_t b0 = hi ? prmt<0x5410>(x[0], x[1]) : prmt<0x7632>(x[0], x[1]);
        const uint32_t b1 = hi ? prmt<0x5410>(x[2], x[3]) : prmt<0x7632>(x[2], x[3]);
        uint32_t m01 = 0u, m89 = 0u;
        if (MASK) {
            const uint32_t r = msk >> (2 * tq);
            m01 = ((r & 1u) ? 0x0000ffffu : 0u) | ((r & 2u) ? 0xffff0000u : 0u);
            m89 = ((r & 0x100u) ? 0x0000ffffu : 0u) | ((r & 0x200u) ? 0xffff0000u : 0u);
        }
        if constexpr (C::Q8) {
            // the value columns are permuted (see q8_value_col): a 32-bit word at
            // byte 32u + 4gq of a row holds columns gq and gq + 8 of m-tiles 2u, 2u + 1
            const int r0 = 2 * tq, r1 = r0 + 1, r8 = r0 + 8, r9 = r0 + 9;
            const int cwb = wq * C::HPW * C::R;  // first byte column of the warp's private columns
            static_assert(C::KSP % 2 == 0, "pairs of m-tiles");
#pragma unroll
            for (int u = 0; u < 4 + C::KSP / 2; ++u) {
                const int cb = u < 4 ? 32 * u + 4 * gq : cwb + 32 * (u - 4) + 4 * gq;
                const uint8_t *t = st + (u < 4 ? 0 : C::S_BYTES) + (cb & 15);
                const int ch = cb >> 4;
                uint32_t a[4], a2[4];
                q8_pair_frags<MASK>(lds_u32(t + box_chunk_rows<kTS>(r0, ch)), lds_u32(t + box_chunk_rows<kTS>(r1, ch)),
                                    lds_u32(t + box_chunk_rows<kTS>(r8, ch)), lds_u32(t + box_chunk_rows<kTS>(r9, ch)),
                                    m01, m89, a, a2);
                if (u < 4) {
                    mma_f16_16816(accS[(2 * u) & 7], a, b0, b1);
                    mma_f16_16816(accS[(2 * u + 1) & 7], a2, b0, b1);
                } else {
                    mma_f16_16816(accR[(2 * (u - 4)) % C::KSP], a, b0, b1);
                    mma_f16_16816(accR[(2 * (u - 4) + 1) % C::KSP], a2, b0, b1);
                }
            }
        } else {
            const uint32_t base = smem_u32(st);
#pragma unroll
            for (int t = 0; t < 8 + C::KSP; ++t) {
                uint32_t a[4];
                ldmatrix_x4_trans(base + (t < 8 ? at_step(ovs, t) : private_at(ovr, t - 8)), a[0], a[1], a[2], a[3]);
                if (MASK) { a[0] &= m01; a[1] &= m01; a[2] &= m89; a[3] &= m89; }
                if (t < 8) mma_bf16_16816(accS[t & 7], a, b0, b1);
                else mma_bf16_16816(accR[t < 8 ? 0 : t - 8], a, b0, b1);
            }
        }
    }

    // The warp's states to the CTAs that own its heads: state `from` of recv
    // [NG CL][H / CL][WS], from = grp CL + rank.
    __device__ __forceinline__ void send(const WinParams &P, const float *recv, uint64_t *arrived, int from, int CL) const {
        const int HC = C::H / CL;  // heads per owner
        auto at = [&](int h) { return mapa_addr(smem_u32(recv + ((size_t)from * HC + h % HC) * C::WS), h / HC); };
#pragma unroll
        for (int i = 0; i < C::NH; ++i) {
            float x = l[i];
#pragma unroll
            for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            const uint32_t a = at(head(i)) + C::W * 4;
            if (j == 0) {
                st_cluster_f32(a, m[i]);
                st_cluster_f32(a + 4, x);
            }
        }
        // accumulator columns n and 4 + n are added; lanes with tq < 2 hold heads
        // 2tq, 2tq + 1 (of the private rows, those of their own heads)
        const int h0 = wq * C::HPW + 2 * (tq & 1);
        const uint32_t base[2] = {at(h0) + 4u * gq, at(h0 + 1) + 4u * gq};
        const float fs = C::Q8 ? P.sc.y : 1.f, fr = C::Q8 ? P.sc.w : 1.f;
        float v[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[t][e] = (accS[t][e] + __shfl_xor_sync(0xffffffffu, accS[t][e], 2)) * fs;
        constexpr int U = C::R / 8;  // units of eight private columns of a head
        float u[2][U];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float a;
                if constexpr (C::Q8) {
                    a = 0.f;  // (other columns, below)
                } else {
                    const int x = e * U + i, y = (2 + e) * U + i;  // the unit in heads e and 2 + e
                    a = (tq & 1) ? accR[y >> 1][2 * (y & 1) + e] : accR[x >> 1][2 * (x & 1) + e];
                    a += __shfl_xor_sync(0xffffffffu, a, 2);
                }
                u[e][i] = a * fr;
            }
        if (!C::Q8 && tq < 2) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    st_cluster_f32(base[e] + 4 * (16 * t), v[t][e]);
                    st_cluster_f32(base[e] + 4 * (16 * t + 8), v[t][2 + e]);
                }
#pragma unroll
                for (int i = 0; i < U; ++i) st_cluster_f32(base[e] + 4 * (C::DH + 8 * i), u[e][i]);
            }
        }
        if constexpr (C::Q8) {
            // a block of 32 value columns holds columns 4gq + x in m-tile x >> 1,
            // register pair x & 1 (q8_value_col)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (tq < 2) st_cluster_f32(base[e] + 4 * (32 * k + 3 * gq + x), v[2 * k + (x >> 1)][2 * (x & 1) + e]);
#pragma unroll
            for (int k = 0; k < C::KSP / 2; ++k) {
                const int c = 32 * k + 4 * gq, n = c / C::R;  // four columns of one head
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float a = (n & 1) ? accR[2 * k + (x >> 1)][2 * (x & 1) + 1] : accR[2 * k + (x >> 1)][2 * (x & 1)];
                    const float r = (a + __shfl_xor_sync(0xffffffffu, a, 2)) * fr;
                    if (tq == (n >> 1))
                        st_cluster_f32(((n & 1) ? base[1] : base[0]) + 4 * (C::DH + c + x - n * C::R - gq), r);
                }
            }
        }
        __syncwarp();
        const int o0 = wq * C::HPW / HC, o1 = (wq * C::HPW + C::HPW - 1) / HC;  // owners of these heads
        if (lane <= o1 - o0) arrive_cluster(mapa_rank(arrived, o0 + lane));
    }
};

// The copying warp: every slot of the CTA's segments in order, each as soon as
// the ring has room.  Page ids come 32 at a time, one per lane.
template <class C>
__device__ __forceinline__ void copy_tiles(const WinMaps &M, const WinParams &P, uint8_t *smem, int rank, int CL, int cid,
                                           int NC) {
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = reinterpret_cast<uint64_t *>(smem + C::OFF_EMPTY);
    int *okf = reinterpret_cast<int *>(smem + C::OFF_OK);
    const int lane = threadIdx.x & 31;
    // the cache streams through once per step: evict it from L2 first
    const uint64_t pol = l2_evict_first_policy();
    int slot = 0, room = C::SLOTS;
    uint32_t half = 0, old = 0;  // half turns issued, and how many of them are known to be free again
    uint32_t ones = 0;           // bit i: the last half turn with number i mod 32 took one slot
    bool ok_all = true;
    // the n key (value) halves of a turn, at pool rows y
    auto put = [&](bool key, int n, const int (&y)[2], const bool (&ok)[2]) {
        while (room < n && ok_all) {
            ok_all = __all_sync(0xffffffffu, mbar_wait(&empty[old % kBars], (old / kBars) & 1));
            room += C::NG == 1 || ((ones >> (old & 31)) & 1u) ? 1 : 2;
            ++old;
        }
        if (!ok_all) return;
        room -= n;
        ones = n == 1 ? ones | (1u << (half & 31)) : ones & ~(1u << (half & 31));
        uint64_t *bar = &full[half % kBars];
        const bool nk = key && P.norm;
        if (lane == 0) mbar_arrive_expect_tx(bar, n * (C::SLOT + (nk ? C::NKB : 0)));
#pragma unroll
        for (int i = 0; i < C::NG; ++i)
            if (i < n) {
                if (lane == 0) {
                    uint8_t *st = smem + slot * C::SLOT;
                    tma_load_3d_hint(st, key ? &M.sk : &M.sv, 0, y[i], 0, bar, pol);
                    tma_load_3d_hint(st + C::S_BYTES, key ? &M.rk : &M.rv, 0, y[i], 0, bar, pol);
                    if (nk) tma_load_3d_hint(smem + C::OFF_NK + slot * C::NKB, &M.nk, 0, y[i], 0, bar, pol);
                }
                if (++slot == C::SLOTS) slot = 0;
            }
        ++half;
    };
    Segment w;
    for (int k = 0; ok_all && w.at(P, k, cid, NC); ++k) {
        const Range rg(w, rank, CL);
        const VirtualRows vr(w.L, P);
        const int32_t *tab = P.page_table + (size_t)(P.req_row ? P.req_row[w.b] : w.b) * P.max_pages;
        int chunk = -1, id = -1;    // this lane's page id: page 32 chunk + lane
        int pidx = 0, in_page = 0;  // page and row in it of cache row `row`
        int32_t row = -2;
        for (int32_t t = rg.t0; t < rg.t1 && ok_all; t += C::NG * kTS) {
            const int n = C::NG == 2 && rg.t1 - t > kTS ? 2 : 1;
            int y[2] = {0, 0};
            bool ok[2] = {false, false};
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i < n) {
                    const int32_t r = vr.row(t + kTS * i);
                    if (r == row + kTS) {  // the next tile of the same run
                        in_page += kTS;
                        if (in_page >= P.page_size) {
                            in_page = 0;
                            ++pidx;
                        }
                    } else {
                        pidx = r / P.page_size;
                        in_page = r - pidx * P.page_size;
                    }
                    row = r;
                    if ((pidx >> 5) != chunk) {
                        chunk = pidx >> 5;
                        const int at = chunk * 32 + lane;
                        id = at < P.max_pages ? tab[at] : -1;
                    }
                    const int page = __shfl_sync(0xffffffffu, id, pidx & 31);
                    ok[i] = page >= 0 && page < P.num_pages;
                    if (!ok[i] && lane == 0) status_or(P.status, LRKV_STATUS_BAD_PAGE);
                    y[i] = ok[i] ? page * P.page_size + in_page : 0;  // (the heads' warps mask the tile)
                }
            // (published to the heads' warps by the key halves' barrier; a word is
            // rewritten kBars half turns later, when they are long past it)
            if (lane == 0) okf[half % kBars] = (ok[0] ? 1 : 0) | (ok[1] ? 2 : 0);
            put(true, n, y, ok);
            put(false, n, y, ok);
        }
    }
    if (!ok_all && lane == 0) status_or(P.status, LRKV_STATUS_TIMEOUT);
    // every copy has landed before the CTA can leave
    for (uint32_t k = old; k < half; ++k) mbar_wait(&full[k % kBars], (k / kBars) & 1);
}

// Part of p = q B_K[h]: channels d0 .. d0 + 128 / N - 1, into scr [R].  Lane
// o + 8 s (octet o < R / 8 of columns, slice s of the four) has the rows of B_K of
// its slice in flight at once; shuffles add the slices.
template <class C, int N>
__device__ __forceinline__ void private_part(const WinParams &P, int b, int h, int d0, float *scr) {
    constexpr int ROWS = 32 / N;
    const int lane = threadIdx.x & 31, o = lane & 7, sl = lane >> 3;
    const int oc = 8 * o < C::R ? 8 * o : 0;  // (lanes past the last octet repeat the first)
    const __nv_bfloat16 *qr = P.q + ((size_t)b * C::H + h) * C::DH + d0 + ROWS * sl;
    const __nv_bfloat16 *br = P.B_K + ((size_t)h * C::DH + d0 + ROWS * sl) * C::R + oc;
    uint4 qv[ROWS / 8], bv[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS / 8; ++k) qv[k] = *reinterpret_cast<const uint4 *>(qr + 8 * k);
#pragma unroll
    for (int e = 0; e < ROWS; ++e) bv[e] = __ldg(reinterpret_cast<const uint4 *>(br + e * C::R));
    uint64_t acc2[4] = {0, 0, 0, 0};  // pairs of columns
#pragma unroll
    for (int e = 0; e < ROWS; ++e) {
        const uint4 &q4 = qv[e >> 3];
        const uint32_t qw = ((e >> 1) & 3) == 0 ? q4.x : ((e >> 1) & 3) == 1 ? q4.y : ((e >> 1) & 3) == 2 ? q4.z : q4.w;
        const float qf = (e & 1) ? bf16hi(qw) : bf16lo(qw);
        const uint32_t bw[4] = {bv[e].x, bv[e].y, bv[e].z, bv[e].w};
        const uint64_t q2 = f32x2(qf, qf);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc2[c] = f32x2_fma(q2, f32x2(bf16lo(bw[c]), bf16hi(bw[c])), acc2[c]);
    }
    float acc[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) f32x2_unpack(acc2[c], acc[2 * c], acc[2 * c + 1]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], 8);
        acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], 16);
    }
    if (sl == 0 && 8 * o < C::R) {
        float4 *dst = reinterpret_cast<float4 *>(scr + 8 * o);
        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
}

// The private queries of request b, this CTA's H / CL heads, in parts (scr
// [H / CL][N][R]): every head takes N warps, N = 4, 2 or 1 as the CTA has two,
// four or more heads.
template <class C>
__device__ __forceinline__ void private_sums(const WinParams &P, int b, float *scr, int rank, int CL) {
    const int warp = threadIdx.x >> 5, HC = C::H / CL, h0 = rank * HC;
    if (HC == 2) {
        private_part<C, 4>(P, b, h0 + (warp >> 2), 32 * (warp & 3), scr + warp * C::R);
    } else if (HC == 4) {
        private_part<C, 2>(P, b, h0 + (warp >> 1), 64 * (warp & 1), scr + warp * C::R);
    } else {
#pragma unroll 1
        for (int h = warp; h < HC; h += C::NCW) private_part<C, 1>(P, b, h0 + h, 0, scr + h * C::R);
    }
}

// Sum the parts (after a heads_sync), a head per warp, and send them to every CTA
// of the cluster: ph [H][R] gets p rounded, pl the remainders, in a fixed order
// of sums; for an 8-bit cache after the exact power-of-two scaling that brings
// the head's largest |value| into [2^14, 2^15), whose inverse goes to psc [H].
template <class C>
__device__ __forceinline__ void private_send(const float *scr, uint16_t *ph, uint16_t *pl, float *psc, uint64_t *begun,
                                             int rank, int CL) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, HC = C::H / CL, N = HC >= C::NCW ? 1 : C::NCW / HC;
    for (int hh = warp; hh < HC; hh += C::NCW) {
        const int h = rank * HC + hh;
        const bool on = 2 * lane < C::R;
        float y0 = 0.f, y1 = 0.f;
        if (on)
            for (int k = 0; k < N; ++k) {
                const float2 x = *reinterpret_cast<const float2 *>(scr + (hh * N + k) * C::R + 2 * lane);
                y0 += x.x;
                y1 += x.y;
            }
        float back = 1.f;
        if constexpr (C::Q8) {
            float mp = fmaxf(fabsf(y0), fabsf(y1));
#pragma unroll
            for (int k = 16; k; k >>= 1) mp = fmaxf(mp, __shfl_xor_sync(0xffffffffu, mp, k));
            const int ep = f16_range_shift(mp);
            y0 *= exp2i(ep);
            y1 *= exp2i(ep);
            back = exp2i(-ep);
        }
        const uint32_t hw = C::Q8 ? pack_f16(y0, y1) : pack_bf16(y0, y1);
        uint32_t lw;
        if constexpr (C::Q8) {
            const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&hw));
            lw = pack_f16(y0 - r.x, y1 - r.y);
        } else {
            lw = pack_bf16(y0 - bf16lo(hw), y1 - bf16hi(hw));
        }
        const uint32_t ah = smem_u32(ph + h * C::R + 2 * lane), al = smem_u32(pl + h * C::R + 2 * lane);
        for (int k = 0; k < CL; ++k) {
            if (on) {
                st_cluster_u32(mapa_addr(ah, k), hw);
                st_cluster_u32(mapa_addr(al, k), lw);
            }
            if (C::Q8 && lane == 0) st_cluster_f32(mapa_rank(psc + h, k), back);
        }
        __syncwarp();
        if (lane < CL) arrive_cluster(mapa_rank(begun, lane));
    }
}

// The states of the heads this CTA owns are all in recv [NS][HC][WS] (NS = NG CL
// states, HC = H / CL heads): merge them and store the outputs of a whole
// request, or state `slot` for the combine.  bv: the row of B_V of this thread's
// first output, loaded beforehand.
template <class C>
__device__ __forceinline__ void merge_owned(const WinParams &P, int b, int64_t slot, float *recv, float *wts,
                                            const uint4 (&bv)[C::R / 8], int rank, int CL) {
    const int tid = threadIdx.x, HC = C::H / CL, NS = C::NG * CL, h0 = rank * HC;
    static_assert(C::H * C::NG == 32, "a thread of the first warp per weight");
    if (tid < 32) {  // weight of state k of head hh; of a whole request's, divided by the sum
        const int hh = tid / NS, k = tid % NS;
        const float2 s = *reinterpret_cast<const float2 *>(recv + (k * HC + hh) * C::WS + C::W);
        float M = s.x;
        for (int o = 1; o < NS; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float x = s.x == -INFINITY ? 0.f : exp2f(s.x - M);
        float L = x * s.y;
        for (int o = 1; o < NS; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        wts[tid] = P.splits > 1 ? x : L > 0.f ? x / L : 0.f;
        if (P.splits > 1 && k == 0)
            *reinterpret_cast<float2 *>(P.ml + (slot * C::H + h0 + hh) * 2) = make_float2(M, L);
    }
    heads_sync();
    auto merged = [&](int hh, int c) {
        float a = 0.f;
#pragma unroll 8
        for (int k = 0; k < NS; ++k) a = fmaf(wts[hh * NS + k], recv[(k * HC + hh) * C::WS + c], a);
        return a;
    };
    if (P.splits > 1) {
        for (int e = tid; e < HC * C::W; e += C::NT)
            P.acc[(slot * C::H + h0) * C::W + e] = merged(e / C::W, e % C::W);
        return;
    }
    // the private columns, merged in place over the first state's (each read here only)
    for (int e = tid; e < HC * C::R; e += C::NT)
        recv[(e / C::R) * C::WS + C::DH + e % C::R] = merged(e / C::R, C::DH + e % C::R);
    heads_sync();
    // out[b, h] = accS / L + (accR / L) B_V[h]^T, a row of B_V[h] per thread
    for (int e = tid; e < HC * C::DH; e += C::NT) {
        const int hh = e / C::DH, d = e % C::DH, h = h0 + hh;
        uint4 y[C::R / 8];
#pragma unroll
        for (int k = 0; k < C::R / 8; ++k)
            y[k] = e == tid ? bv[k] : __ldg(reinterpret_cast<const uint4 *>(P.B_V + ((size_t)h * C::DH + d) * C::R) + k);
        float v = merged(hh, d);
        const float *r = recv + hh * C::WS + C::DH;
#pragma unroll
        for (int k = 0; k < C::R / 8; ++k, r += 8) {
            const float4 r0 = *reinterpret_cast<const float4 *>(r), r1 = *reinterpret_cast<const float4 *>(r + 4);
            v = fmaf(r0.x, bf16lo(y[k].x), v); v = fmaf(r0.y, bf16hi(y[k].x), v);
            v = fmaf(r0.z, bf16lo(y[k].y), v); v = fmaf(r0.w, bf16hi(y[k].y), v);
            v = fmaf(r1.x, bf16lo(y[k].z), v); v = fmaf(r1.y, bf16hi(y[k].z), v);
            v = fmaf(r1.z, bf16lo(y[k].w), v); v = fmaf(r1.w, bf16hi(y[k].w), v);
        }
        P.out[((size_t)b * C::H + h) * C::DH + d] = __float2bfloat16_rn(v);
    }
}

}  // namespace

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    decode_window_kernel(const __grid_constant__ WinMaps M, const __grid_constant__ WinParams P) {
    extern __shared__ uint8_t smem_raw[];
    // the same offset in every CTA of a cluster (the base of dynamic shared memory is)
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = reinterpret_cast<uint64_t *>(smem + C::OFF_EMPTY);
    // begun: a segment's private queries are in ph, pl; arrived: the states of the
    // owned heads are in recv; freed: every CTA is done with a segment
    uint64_t *begun = reinterpret_cast<uint64_t *>(smem + C::OFF_CB), *arrived = begun + 1, *freed = begun + 2;
    const int *okf = reinterpret_cast<const int *>(smem + C::OFF_OK);
    uint16_t *ph = reinterpret_cast<uint16_t *>(smem + C::OFF_P), *pl = ph + C::H * C::R;
    float *psc = reinterpret_cast<float *>(smem + C::OFF_PSC);
    float *recv = reinterpret_cast<float *>(smem + C::OFF_RECV);
    float *wts = reinterpret_cast<float *>(smem + C::OFF_WTS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int CL = cluster_nctarank(), rank = cluster_ctarank();
    const int NC = gridDim.x / CL, cid = blockIdx.x / CL, HC = C::H / CL;

    if (tid < kBars) {
        mbar_init(&full[tid], 1);
        mbar_init(&empty[tid], C::NCW);
    } else if (tid == 32) {
        mbar_init(begun, C::H);
        mbar_init(arrived, C::NG * CL * max(1, HC / C::HPW));  // the warps of each CTA that hold such heads
        mbar_init(freed, CL);
    } else if (tid == 64) {
        prefetch_tensormap(&M.sk);
        prefetch_tensormap(&M.sv);
        prefetch_tensormap(&M.rk);
        prefetch_tensormap(&M.rv);
        if (P.norm) prefetch_tensormap(&M.nk);
    }
    if (tid <= 32) fence_barrier_init();
    // warm L2 with the owned heads' bases while the predecessor finishes
    prefetch_l2(P.B_K + rank * HC * C::DH * C::R, (size_t)HC * C::DH * C::R * 2, tid, C::THREADS);
    if (P.splits == 1) prefetch_l2(P.B_V + rank * HC * C::DH * C::R, (size_t)HC * C::DH * C::R * 2, tid, C::THREADS);
    __syncthreads();
    // no peer's shared memory is used before its CTA has come this far (waited
    // for before the first private queries are sent)
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    pdl_wait();
    pdl_launch_dependents();

    if (warp >= C::NCW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_COPY));
        if (warp == C::NCW) copy_tiles<C>(M, P, smem, rank, CL, cid, NC);
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        return;
    }

    // ---- the heads' warps
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_HEADS));
    HeadState<C> hs;
    Segment w;
    bool have = w.at(P, 0, cid, NC), timed_out = false;
    uint32_t half = 0;  // half turns consumed
    int slot = 0;       // the next one's first slot
    if (have) {
        private_sums<C>(P, w.b, recv, rank, CL);
        hs.begin_shared(P, w.b);
        heads_sync();
    }
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (have) private_send<C>(recv, ph, pl, psc, begun, rank, CL);
    for (int turn = 0; have; ++turn) {  // (all CTAs of a cluster walk the same segments)
        auto wait_cluster = [&](uint64_t *bar, int n) {
            if (!mbar_wait_cluster(bar, n & 1) && lane == 0) status_or(P.status, LRKV_STATUS_TIMEOUT);
        };
        wait_cluster(begun, turn);
        hs.begin_private(P, (hs.hi ? ph : pl) + hs.wq * C::HPW * C::R, psc + hs.wq * C::HPW);
        const VirtualRows vr(w.L, P);
        const Range rg(w, rank, CL);
        if (vr.total == 0 && rank == 0 && tid == 0) status_or(P.status, LRKV_STATUS_BAD_SEQLEN);
        auto wait_half = [&](uint32_t h) {
            if (!__all_sync(0xffffffffu, mbar_wait(&full[h % kBars], (h / kBars) & 1))) {
                if (lane == 0) status_or(P.status, LRKV_STATUS_TIMEOUT);
                timed_out = true;
            }
            return !timed_out;
        };
        auto release = [&](uint32_t h) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[h % kBars]);
        };
        for (int t = rg.t0; t < rg.t1 && !timed_out; t += C::NG * kTS, half += 2) {
            // the key halves of this turn's n tiles, then the value halves
            const int n = C::NG == 2 && rg.t1 - t > kTS ? 2 : 1;
            int ks = slot + hs.grp, vs = slot + n + hs.grp;
            ks -= ks >= C::SLOTS ? C::SLOTS : 0;
            vs -= vs >= C::SLOTS ? C::SLOTS : 0;
            slot += 2 * n;
            slot -= slot >= C::SLOTS ? C::SLOTS : 0;
            if (!wait_half(half)) break;
            if (C::NG == 2 && hs.grp >= n) {  // (the last turn may have one tile)
                release(half);
                if (!wait_half(half + 1)) break;
                release(half + 1);
                continue;
            }
            // rows of the tile that are attended: those of the segment, and of them
            // the sinks and the window
            const int32_t v = t + kTS * hs.grp, row = vr.row(v);
            uint32_t msk = 0xffffu;
            if (v < w.va || v + kTS > w.vb || (row < vr.first && row + kTS > vr.sinks)) {
                auto below = [](int32_t x) -> uint32_t { return x >= kTS ? 0xffffu : x <= 0 ? 0u : (1u << x) - 1u; };
                msk = below(w.vb - v) & ~below(w.va - v) & (below(vr.sinks - row) | ~below(vr.first - row)) & 0xffffu;
            }
            if (((okf[half % kBars] >> hs.grp) & 1) == 0) msk = 0u;
            float s[C::NH];
            hs.scores(P, smem + ks * C::SLOT, smem + C::OFF_NK + ks * C::NKB, (msk >> hs.j) & 1u, s);
            release(half);
            hs.softmax(s);
            if (!wait_half(half + 1)) break;
            if (msk == 0xffffu) hs.template values<false>(smem + vs * C::SLOT, s, msk);
            else hs.template values<true>(smem + vs * C::SLOT, s, msk);
            release(half + 1);
        }
        // ---- the states, to the owners of their heads (whose recv is free: they
        // have sent this segment's private queries, which were summed there)
        hs.send(P, recv, arrived, hs.grp * CL + rank, CL);
        uint4 bv[C::R / 8];  // the row of B_V of this thread's first output, in flight while the states travel
#pragma unroll
        for (int k = 0; k < C::R / 8; ++k)
            bv[k] = __ldg(reinterpret_cast<const uint4 *>(
                              P.B_V + (size_t)min(rank * HC * C::DH + tid, C::H * C::DH - 1) * C::R) + k);
        wait_cluster(arrived, turn);
        merge_owned<C>(P, w.b, cid + (int64_t)turn * NC, recv, wts, bv, rank, CL);
        have = w.at(P, turn + 1, cid, NC);
        if (have) {
            heads_sync();  // recv and this CTA's private queries are read
            if (tid < CL) arrive_cluster(mapa_rank(freed, tid));
            private_sums<C>(P, w.b, recv, rank, CL);
            hs.begin_shared(P, w.b);
            heads_sync();
            wait_cluster(freed, turn);
            private_send<C>(recv, ph, pl, psc, begun, rank, CL);
        }
    }
}

// ---------------------------------------------------------------------------
// Combine of a request's splits: block (head, request), a thread per output
// column.  Log-sum-exp merge of the S states, then out = accS / L + (accR / L)
// B_V[h]^T (equation 7).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128) window_combine_kernel(const __nv_bfloat16 *__restrict__ B_V,
                                                             const float *__restrict__ ml, const float *__restrict__ acc,
                                                             int H, int r, int S, __nv_bfloat16 *__restrict__ out) {
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, W = 128 + r;
    __shared__ float wts[32], priv[64];
    // (a weight of the call: complete before the main kernel let this one launch)
    uint4 bv[8];
    const uint4 *row = reinterpret_cast<const uint4 *>(B_V + ((size_t)h * 128 + tid) * r);
#pragma unroll
    for (int k = 0; k < 8; ++k) bv[k] = 8 * k < r ? __ldg(row + k) : make_uint4(0u, 0u, 0u, 0u);
    pdl_wait();
    pdl_launch_dependents();
    const size_t s0 = ((size_t)b * S) * H + h;  // state of split k: s0 + k H
    // this thread's shared column and, of the first r, a private one, eight splits
    // at a time; the first eight are on the way while the weights are formed
    constexpr int N = 8;
    float av[N], ap[N];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float *a = acc + (s0 + (size_t)(k0 + i) * H) * W;
            av[i] = k0 + i < S ? a[tid] : 0.f;
            ap[i] = k0 + i < S && tid < r ? a[128 + tid] : 0.f;
        }
    };
    fetch(0);
    if (tid < 32) {
        const float2 s = tid < S ? *reinterpret_cast<const float2 *>(ml + (s0 + (size_t)tid * H) * 2)
                                 : make_float2(-INFINITY, 0.f);
        float M = s.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float x = s.x == -INFINITY ? 0.f : exp2f(s.x - M);
        float L = x * s.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        wts[tid] = L > 0.f ? x / L : 0.f;
    }
    float v = 0.f, p = 0.f;
    __syncthreads();
    for (int k0 = 0; k0 < S; k0 += N) {  // (weights past S are 0: kMaxSplits is a multiple of N)
        if (k0) fetch(k0);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v = fmaf(wts[k0 + i], av[i], v);
            p = fmaf(wts[k0 + i], ap[i], p);
        }
    }
    if (tid < 64) priv[tid] = tid < r ? p : 0.f;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float *x = priv + 8 * k;
        v = fmaf(x[0], bf16lo(bv[k].x), v); v = fmaf(x[1], bf16hi(bv[k].x), v);
        v = fmaf(x[2], bf16lo(bv[k].y), v); v = fmaf(x[3], bf16hi(bv[k].y), v);
        v = fmaf(x[4], bf16lo(bv[k].z), v); v = fmaf(x[5], bf16hi(bv[k].z), v);
        v = fmaf(x[6], bf16lo(bv[k].w), v); v = fmaf(x[7], bf16hi(bv[k].w), v);
    }
    out[((size_t)b * H + h) * 128 + tid] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Clusters of CL CTAs that the current device holds at once (one CTA fills an SM).
static int active_clusters(const void *kern, int smem, int nthreads, int CL, cudaError_t *err) {
    struct Key {
        const void *kern;
        int dev, CL, n;
    };
    static std::mutex mu;
    static Key known[512];  // (past these the query is simply made each time)
    static int count = 0;
    int dev = 0;
    if ((*err = cudaGetDevice(&dev)) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < count; ++i)
        if (known[i].kern == kern && known[i].dev == dev && known[i].CL == CL) return known[i].n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CL);
    cfg.blockDim = dim3(nthreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if ((*err = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return 0;
    if (count < 512) known[count++] = {kern, dev, CL, n};
    return n;
}

// The layout with the least estimated time.  A CTA takes a tile (tile_bytes) in
// 12 ns per KB of bf16 rows, 34 ns per KB of 8-bit codes (0.67 us and 1.0 us for
// 16 heads, r = 48); a segment costs a cluster fixed[] us besides (private
// queries, start of the ring, the states' way to their owners; measured for
// segments of a few tiles), a combine 4 us, and nothing is faster than the copy
// bandwidth.  A split without a workspace at hand (unsplit_below: 25 us) costs the
// caller another call and an allocation: it is chosen only where both layouts
// take longer than that.  Measured at 16 heads, r = 48, against this rule's choice:
//   16 requests, window 1024:  CL 1, 2, 4, 8 in 58.5, 33.9, 22.1, 31.0 us (eight
//     CTAs a cluster: 15 clusters fit the GPU at once, so one request waits)
//   64 requests, window 1024:  61.5, 45.5, 51.5, 76.9 us
//   1 request, window 8000:    CL 8 unsplit 51.1 us, split over 15 clusters 18.4 us
//   1 request, window 1024:    unsplit 13.4 us, split 10.8; 4 requests, window
//     2048: 20.0, 16.3; 16 requests, window 1024: 21.8, 21.0; 40, window 2048:
//     60.8, 57.1 (a combine taken as 2 us: 12 requests, window 2048: 25.1 for 23.3)
// `rows`: visible rows of the longest request; active[i]: clusters of 1 << i CTAs
// that the GPU holds at once.
static WindowLayout window_plan(int B, int64_t rows, double tile_bytes, bool q8, int most_splits, double unsplit_below,
                                const int (&active)[4]) {
    static const double fixed[4] = {17., 12., 9., 8.}, combine = 4.;
    const int64_t tiles = (rows + kTS - 1) / kTS;
    const double tile_us = tile_bytes / 1024. * (q8 ? 0.034 : 0.012);
    const double hbm_us = (double)B * tiles * tile_bytes / 6.5e6;
    WindowLayout best{1, 1, 1};
    double least = 1e300;
    auto consider = [&](int i, int64_t S) {
        const int64_t CL = 1 << i, used = std::min<int64_t>((int64_t)B * S, active[i]);
        const int64_t rounds = ((int64_t)B * S + used - 1) / used, per_cta = ((tiles + S - 1) / S + CL - 1) / CL;
        const double work = rounds * (per_cta * tile_us + fixed[i]);
        // (where the memory's rate decides, the layout with the fewest segments)
        double t = std::max(work, hbm_us) + 0.3 * rounds * fixed[i];
        if (S > 1) t = std::max(t + combine, unsplit_below);
        if (t < least) {
            least = t;
            best = {(int)CL, (int)used, (int)S};
        }
        return per_cta;
    };
    for (int i = 0; i < 4; ++i)
        if (active[i] > 0) consider(i, 1);
    for (int i = 0; i < 4; ++i) {
        // (the least that splits could take)
        if (active[i] < 1 || std::max(1.3 * fixed[i] + tile_us + combine, unsplit_below) >= least) continue;
        const int64_t smax = std::min<int64_t>(most_splits, active[i] / B);
        for (int64_t S = 2; S <= smax; ++S)
            if (consider(i, S) == 1) break;  // (more splits take no less)
    }
    return best;
}

// Visible rows of the longest request that a call lays out, tile edges included.
static int64_t planned_rows(int max_seq_len, int window, int sinks) {
    return std::min<int64_t>(max_seq_len, (int64_t)window + sinks) + kTS;
}

// active[i]: clusters of 1 << i CTAs that the GPU holds at once.
template <class C>
static cudaError_t active_cfg(int (&active)[4]) {
    auto kern = decode_window_kernel<C>;
    cudaError_t e = smem_limit_once(kern, C::SMEM);
    for (int i = 0; i < 4 && e == cudaSuccess; ++i)
        active[i] = active_clusters(reinterpret_cast<const void *>(kern), C::SMEM, C::THREADS, 1 << i, &e);
    return e;
}

template <class C>
static cudaError_t plan_cfg(int B, int max_seq_len, int window, int sinks, WindowLayout *plan, int most_splits = kMaxSplits,
                            double unsplit_below = 0.) {
    int active[4];
    const cudaError_t e = active_cfg<C>(active);
    if (e == cudaSuccess)
        *plan = window_plan(B, planned_rows(max_seq_len, window, sinks), 2.0 * C::SLOT, C::Q8, most_splits,
                            unsplit_below, active);
    return e;
}

// The layout of a call within its scratch.
template <class C>
static cudaError_t layout_cfg(const DecodeArgs &a, const void *ws, size_t ws_bytes, WindowLayout *plan) {
    cudaError_t e = plan_cfg<C>(a.B, a.max_seq_len, a.window, a.sinks, plan, kMaxSplits, ws ? 0. : 25.);
    if (e != cudaSuccess) return e;
    if (plan->S > 1 && !ws) return cudaErrorNotSupported;
    if (plan->S > 1 && ws_bytes < (size_t)a.B * plan->S * C::H * (2 + C::W) * sizeof(float))  // (a prefill's workspace)
        e = plan_cfg<C>(a.B, a.max_seq_len, a.window, a.sinks, plan, 1);
    return e;
}

template <class C>
static cudaError_t launch_cfg(const DecodeArgs &a, void *ws, const WindowLayout &plan) {
    constexpr int H = C::H, R = C::R, NGRP = C::NGRP;
    constexpr bool Q8 = C::Q8;
    const auto &c = a.cache;
    const int64_t pool_rows = (int64_t)c.num_pages * c.page_size;
    WinMaps maps;
    if (!make_map(&maps.sk, c.S_K, pool_rows, 128 * NGRP, C::EB, 0, false, kTS) ||
        !make_map(&maps.sv, c.S_V, pool_rows, 128 * NGRP, C::EB, 0, false, kTS) ||
        !make_map(&maps.rk, c.R_K, pool_rows, H * R, C::EB, 0, false, kTS) ||
        !make_map(&maps.rv, c.R_V, pool_rows, H * R, C::EB, 0, false, kTS) ||
        (c.N_K && !make_row_map(&maps.nk, c.N_K, pool_rows, H, 2, kTS)))
        return cudaErrorInvalidValue;
    const size_t states = (size_t)a.B * plan.S * H;
    WinParams P;
    P.q = static_cast<const __nv_bfloat16 *>(a.q);
    P.B_K = static_cast<const __nv_bfloat16 *>(a.B_K);
    P.B_V = static_cast<const __nv_bfloat16 *>(a.B_V);
    P.out = static_cast<__nv_bfloat16 *>(a.out);
    P.seq_lens = a.seq_lens;
    P.page_table = a.page_table;
    P.req_row = a.req_row;
    P.B = a.B;
    P.max_pages = a.max_pages;
    P.num_pages = c.num_pages;
    P.page_size = c.page_size;
    P.max_len = decode_max_len(a);
    P.window = a.window;
    P.sinks = a.sinks;
    P.splits = plan.S;
    P.norm = c.N_K != nullptr;
    P.scale_log2 = 1.4426950408889634f / sqrtf(128.f);
    P.sc = Q8 ? make_float4(c.scale[0], c.scale[1], c.scale[2], c.scale[3]) : make_float4(1.f, 1.f, 1.f, 1.f);
    P.acc = static_cast<float *>(ws);
    P.ml = P.acc + states * C::W;
    P.status = a.status;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.NC * plan.CL);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = plan.CL;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // (the kernel's shared-memory limit was set for the layout)
    cudaError_t e = cudaLaunchKernelEx(&cfg, decode_window_kernel<C>, maps, P);
    if (e == cudaSuccess && plan.S > 1)
        e = launch_pdl(window_combine_kernel, dim3(H, a.B), dim3(128), 0, a.stream, P.B_V, (const float *)P.ml,
                       (const float *)P.acc, H, R, plan.S, P.out);
    return e;
}

// f(configuration) of a cache's shape.
template <typename F>
static cudaError_t with_cfg(const lrkv_cache_t &c, F &&f) {
    if (cache_groups(c) == 2) {
#define X(h, rr) \
        if (c.H == h && c.r == rr) return f(WinCfg<h, rr, false, 2>{});
        LRKV_FAST_SHAPES_G2(X)
#undef X
        return cudaErrorInvalidValue;
    }
    const bool q8 = c.dtype == LRKV_FP8_E4M3;
#define X(h, rr)                                                                                            \
    if (c.H == h && c.r == rr) return q8 ? f(WinCfg<h, rr, true, 1>{}) : f(WinCfg<h, rr, false, 1>{});
    LRKV_FAST_SHAPES(X)
#undef X
    return cudaErrorInvalidValue;
}

cudaError_t window_layout(const DecodeArgs &a, const void *ws, size_t ws_bytes, WindowLayout *layout) {
    return with_cfg(a.cache, [&](auto cfg) { return layout_cfg<decltype(cfg)>(a, ws, ws_bytes, layout); });
}

cudaError_t launch_window_fast(const DecodeArgs &a, void *ws, const WindowLayout &layout) {
    return with_cfg(a.cache, [&](auto cfg) { return launch_cfg<decltype(cfg)>(a, ws, layout); });
}

// Bytes that the states of split requests need at most, in this call and in every
// call with fewer requests or shorter lengths or windows (0 for shapes that this
// kernel does not cover).  The number of splits that window_plan chooses rises and
// falls with each size (16 heads, r = 48, window 2048: 364 KB for 16 requests, none
// for 24), so this counts what bounds it: the clusters that the GPU holds at once,
// kMaxSplits for a request, and its tiles.  About 3 MB at most.  Of the two group counts
// of a shape it takes the larger need.
size_t window_state_bytes(int B, int H, int r, int max_seq_len, int window, int sinks, int dtype) {
    int most = 0;  // clusters at once
    auto add = [&](auto cfg) {
        int active[4];
        if (active_cfg<decltype(cfg)>(active) != cudaSuccess) cudaGetLastError();  // (no device: sizing queries only)
        else most = std::max({most, active[0], active[1], active[2], active[3]});
    };
#define X(h, rr)                                              \
    if (H == h && r == rr) {                                  \
        if (dtype == LRKV_FP8_E4M3) add(WinCfg<h, rr, true, 1>{}); \
        else add(WinCfg<h, rr, false, 1>{});                  \
    }
    if (dtype != LRKV_F32) { LRKV_FAST_SHAPES(X) }
#undef X
#define X(h, rr) \
    if (H == h && r == rr) add(WinCfg<h, rr, false, 2>{});
    if (dtype == LRKV_BF16) { LRKV_FAST_SHAPES_G2(X) }
#undef X
    const int64_t tiles = (planned_rows(max_seq_len, window, sinks) + kTS - 1) / kTS;
    const int64_t states = std::min<int64_t>(most, B * std::min<int64_t>(kMaxSplits, tiles));
    return (size_t)states * H * (128 + r + 2) * sizeof(float);
}

}  // namespace lrkv
