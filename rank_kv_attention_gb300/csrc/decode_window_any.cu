// Decode through a sliding window with sinks for the shapes and element types
// that the tensor-core kernel (decode_window.cu) does not cover: fp32 caches, any
// head count, widths up to 256.
//
// One launch: a cluster of CL CTAs takes one (request, head) and its CTAs take
// the visible rows in turn.  Eight lanes (a `group`) take a row at a time, each
// 16 bytes of it (8 of 8-bit codes) per step; every group runs its own online
// softmax (running maximum, sum, shared and private value accumulators), so no
// barrier sits in the row loop.  States are merged by the log-sum-exp rule: the
// four groups of a warp by shuffles, the eight warps in shared memory, the CTAs
// of the cluster through distributed shared memory; then the private part is
// expanded by B_V[h] (equation 7).  All in fp32.
//
// Bound by the latency of the row loads: a row's loads (keys and values, shared
// and private) are all issued before its score, and each group has two rows in
// flight.  Every head reads the shared rows again (out of L2).  6 fp32 requests of
// 8 heads, window 500 (2.9 MB): 10.5 us in a graph, where the generic split kernel and
// its combine took 54 us a call and this takes 20, most of it the call's.
// 16 requests, window 1024, d_h = 128, r = 48: 47 us with 8 heads in bf16 (5.0 at the
// copy bandwidth), 184 with 40 heads (19.9), 106 with 16 heads in fp32 (17.4).  Far
// from the floor: every head's cluster reads the shared rows, and at d_h = 128 a lane
// runs the form for 256 columns with half of its slots empty, at 236 to 255 registers
// (fp32 with d_h and r above 64 spills 696 bytes).
#include <algorithm>

#include "decode_kernels.cuh"
#include "tc_pair.cuh"

namespace lrkv {

namespace {

constexpr int kWarps = 8, kGroups = 4 * kWarps;  // groups of eight lanes per CTA

struct AnyParams {
    const void *q, *S_K, *S_V, *R_K, *R_V, *B_K, *B_V, *N_K;
    void *out;
    const int32_t *seq_lens, *page_table, *req_row;
    int max_pages, num_pages, page_size, max_len, window, sinks;
    int H, d_h, r, s_stride, hpg;  // elements of a token's shared row; heads per shared group
    float scale_log2;
    float4 sc;  // 8-bit cache: pool scales of S_K, S_V, R_K, R_V
    int32_t *status;
};

// V consecutive cache elements, widened.
template <typename TC> struct Chunk;
template <> struct Chunk<float> {
    static constexpr int V = 4;
    float4 x;
    __device__ __forceinline__ void load(const float *p) { x = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void zero() { x = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; }
};
template <> struct Chunk<__nv_bfloat16> {
    static constexpr int V = 8;
    uint4 x;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { x = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { x = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = bf16lo(x.x); v[1] = bf16hi(x.x); v[2] = bf16lo(x.y); v[3] = bf16hi(x.y);
        v[4] = bf16lo(x.z); v[5] = bf16hi(x.z); v[6] = bf16lo(x.w); v[7] = bf16hi(x.w);
    }
};
template <> struct Chunk<uint8_t> {
    static constexpr int V = 8;
    uint2 x;
    __device__ __forceinline__ void load(const uint8_t *p) { x = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void zero() { x = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[2] = {x.x, x.y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t h2 = f16x2_from_e4m3x2((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            v[2 * k] = f.x;
            v[2 * k + 1] = f.y;
        }
    }
};

__device__ __forceinline__ float ld_peer_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// T: query element type; TC: cache element type; NS, NR: chunks of a shared
// (private) row per lane.
template <typename T, typename TC, int NS, int NR>
__global__ void __launch_bounds__(32 * kWarps) decode_window_any_kernel(const __grid_constant__ AnyParams P) {
    constexpr int V = Chunk<TC>::V;
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, li = lane & 7;
    const int CL = cluster_nctarank(), rank = cluster_ctarank();
    const int b = blockIdx.x / CL, h = blockIdx.y;
    const int d_h = P.d_h, r = P.r, W = d_h + r;
    float *qs = sm;                // [d_h] q, then merged shared columns
    float *ps = qs + d_h;          // [r] p, then merged private columns
    float *st = ps + r;            // [kWarps][W + 2] states; partial sums of p before
    float *fin = st + kWarps * (W + 2);  // [W + 2] the CTA's state
    pdl_wait();
    pdl_launch_dependents();
    const int32_t L = P.seq_lens[b];
    const bool valid = L >= 1 && L <= P.max_len;
    if (!valid && rank == 0 && h == 0 && tid == 0) status_or(P.status, LRKV_STATUS_BAD_SEQLEN);
    const VisibleRows vis(valid ? L : 1, P.window, P.sinks);
    const int32_t rows = valid ? L - vis.first + vis.sinks : 0;

    // ---- q and p = q B_K[h] (pool scales folded in): thread (part, column) sums
    // the channels part, part + parts, ...
    const T *q = static_cast<const T *>(P.q) + ((size_t)b * P.H + h) * d_h;
    for (int d = tid; d < d_h; d += 32 * kWarps) qs[d] = Elem<T>::load(q + d);
    __syncthreads();
    {
        const T *B = static_cast<const T *>(P.B_K) + (size_t)h * d_h * r;
        const int parts = 32 * kWarps / r, part = tid / r, k = tid - part * r;  // (r <= 256 threads)
        float a = 0.f;
        if (part < parts)
#pragma unroll 8
            for (int d = part; d < d_h; d += parts) a = fmaf(qs[d], Elem<T>::load(B + (size_t)d * r + k), a);
        if (part < parts) st[part * r + k] = a;
        __syncthreads();
        if (tid < r) {
            float x = 0.f;
            for (int i = 0; i < parts; ++i) x += st[i * r + tid];
            ps[tid] = x;
        }
        __syncthreads();
    }
    float qv[NS][V], pv[NR][V];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int d = (li + 8 * i) * V + e;
            qv[i][e] = d < d_h ? qs[d] * P.sc.x : 0.f;
        }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int k = (li + 8 * i) * V + e;
            pv[i][e] = k < r ? ps[k] * P.sc.z : 0.f;
        }

    // ---- the visible rows, two at a time per group
    float m = -INFINITY, l = 0.f, aS[NS][V], aR[NR][V];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) aS[i][e] = 0.f;
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) aR[i][e] = 0.f;
    const int32_t *pt = P.page_table + (size_t)(P.req_row ? P.req_row[b] : b) * P.max_pages;
    const size_t s_off = (size_t)(h / P.hpg) * d_h;
    const int32_t step = kGroups * CL;
    for (int32_t v0 = rank * kGroups + warp * 4; v0 < rows; v0 += 2 * step) {  // (uniform in the warp)
        Chunk<TC> kS[2][NS], kR[2][NR], vS[2][NS], vR[2][NR];
        bool ok[2];
        float nk[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int32_t v = v0 + (lane >> 3) + u * step;
            ok[u] = v < rows;
            nk[u] = 1.f;
            int64_t prow = 0;
            if (ok[u]) {
                const int32_t j = vis.row(v), page = pt[j / P.page_size];
                ok[u] = page >= 0 && page < P.num_pages;
                if (!ok[u] && li == 0) status_or(P.status, LRKV_STATUS_BAD_PAGE);
                prow = (int64_t)page * P.page_size + j % P.page_size;
            }
            const size_t so = (size_t)prow * P.s_stride + s_off, ro = ((size_t)prow * P.H + h) * r;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int d = (li + 8 * i) * V;
                kS[u][i].zero();
                vS[u][i].zero();
                if (ok[u] && d < d_h) {
                    kS[u][i].load(static_cast<const TC *>(P.S_K) + so + d);
                    vS[u][i].load(static_cast<const TC *>(P.S_V) + so + d);
                }
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int k = (li + 8 * i) * V;
                kR[u][i].zero();
                vR[u][i].zero();
                if (ok[u] && k < r) {
                    kR[u][i].load(static_cast<const TC *>(P.R_K) + ro + k);
                    vR[u][i].load(static_cast<const TC *>(P.R_V) + ro + k);
                }
            }
            if (ok[u] && P.N_K) nk[u] = Elem<T>::load(static_cast<const T *>(P.N_K) + (size_t)prow * P.H + h);
        }
        float s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float a = 0.f, c = 0.f, x[V];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                kS[u][i].get(x);
#pragma unroll
                for (int e = 0; e < V; ++e) a = fmaf(qv[i][e], x[e], a);
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                kR[u][i].get(x);
#pragma unroll
                for (int e = 0; e < V; ++e) c = fmaf(pv[i][e], x[e], c);
            }
            a += c;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
            s[u] = ok[u] ? a * nk[u] * P.scale_log2 : -INFINITY;
        }
        const float mx = fmaxf(m, fmaxf(s[0], s[1]));
        const float al = m == mx ? 1.f : exp2f(m - mx);  // (m = -inf: 0)
        // (a NaN score gives a NaN weight, also while the maximum is still -inf)
        const float e0 = s[0] == -INFINITY ? 0.f : exp2f(s[0] - mx);
        const float e1 = s[1] == -INFINITY ? 0.f : exp2f(s[1] - mx);
        m = mx;
        l = l * al + (e0 + e1);
        float x0[V], x1[V];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            vS[0][i].get(x0);
            vS[1][i].get(x1);
#pragma unroll
            for (int e = 0; e < V; ++e) aS[i][e] = fmaf(e1, x1[e], fmaf(e0, x0[e], aS[i][e] * al));
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            vR[0][i].get(x0);
            vR[1][i].get(x1);
#pragma unroll
            for (int e = 0; e < V; ++e) aR[i][e] = fmaf(e1, x1[e], fmaf(e0, x0[e], aR[i][e] * al));
        }
    }

    // ---- the four groups of the warp
    {
        float M = m;
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float f = m == -INFINITY ? 0.f : exp2f(m - M);
        auto join = [&](float x) {
            x *= f;
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            return x + __shfl_xor_sync(0xffffffffu, x, 16);
        };
        l = join(l);
        float *mine = st + warp * (W + 2);
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float x = join(aS[i][e]);
                const int d = (li + 8 * i) * V + e;
                if (lane < 8 && d < d_h) mine[d] = x;
            }
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float x = join(aR[i][e]);
                const int k = (li + 8 * i) * V + e;
                if (lane < 8 && k < r) mine[d_h + k] = x;
            }
        if (lane == 0) {
            mine[W] = M;
            mine[W + 1] = l;
        }
    }
    __syncthreads();
    // ---- the eight warps, then the CTAs of the cluster (the first one merges)
    auto merge = [&](int n, auto at, float *dst) {  // states at(k) + column
        float M = -INFINITY, Ls = 0.f;
        for (int k = 0; k < n; ++k) M = fmaxf(M, at(k, W));
        // (weight 0 for a state without rows; its sums are 0, or NaN after NaN scores)
        auto weight = [&](int k) {
            const float mk = at(k, W);
            return mk == -INFINITY ? 0.f : exp2f(mk - M);
        };
        for (int k = 0; k < n; ++k) Ls = fmaf(weight(k), at(k, W + 1), Ls);
        for (int c = tid; c < W; c += 32 * kWarps) {
            float a = 0.f;
            for (int k = 0; k < n; ++k) a = fmaf(weight(k), at(k, c), a);
            dst[c] = a;
        }
        if (tid == 0) {
            dst[W] = M;
            dst[W + 1] = Ls;
        }
    };
    merge(kWarps, [&](int k, int c) { return st[k * (W + 2) + c]; }, fin);
    if (CL > 1) {
        cluster_sync_all();
        if (rank == 0) {
            const uint32_t a = smem_u32(fin);
            merge(CL, [&](int k, int c) { return ld_peer_f32(mapa_addr(a, k) + 4 * c); }, st);
        }
        cluster_sync_all();  // no CTA leaves while its state is being read
        if (rank > 0) return;
        fin = st;
    } else {
        __syncthreads();
    }
    // ---- out = accS / L + (accR / L) B_V[h]^T
    const float Ls = fin[W + 1], inv = Ls > 0.f ? 1.f / Ls : 0.f;
    const T *B = static_cast<const T *>(P.B_V) + (size_t)h * d_h * r;
    T *out = static_cast<T *>(P.out) + ((size_t)b * P.H + h) * d_h;
    constexpr int BV = Vec16<T>::N;
    for (int d = tid; d < d_h; d += 32 * kWarps) {
        float a = 0.f;
#pragma unroll 4
        for (int k = 0; k < r; k += BV) {
            float x[BV];
            Vec16<T>::load(B + (size_t)d * r + k, x);
#pragma unroll
            for (int e = 0; e < BV; ++e) a = fmaf(fin[d_h + k + e], x[e], a);
        }
        Elem<T>::store(out + d, (fin[d] * P.sc.y + a * P.sc.w) * inv);
    }
}

template <typename T, typename TC, int NS, int NR>
cudaError_t launch(const AnyParams &P, int B, int CL, cudaStream_t s) {
    const size_t W = P.d_h + P.r;
    const size_t sm = sizeof(float) * (W + std::max<size_t>((kWarps + 1) * (W + 2), 32 * kWarps));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)B * CL, P.H);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = sm;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, decode_window_any_kernel<T, TC, NS, NR>, P);
}

// Chunks per lane: rows of up to 8 `lo` chunks take the small form, others the
// largest (256 elements).
template <typename T, typename TC, int lo, int hi>
cudaError_t launch_sized(const AnyParams &P, int B, int CL, cudaStream_t s) {
    constexpr int n = 8 * lo * Chunk<TC>::V;
    if (P.d_h <= n) return P.r <= n ? launch<T, TC, lo, lo>(P, B, CL, s) : launch<T, TC, lo, hi>(P, B, CL, s);
    return P.r <= n ? launch<T, TC, hi, lo>(P, B, CL, s) : launch<T, TC, hi, hi>(P, B, CL, s);
}

}  // namespace

cudaError_t launch_window_any(const DecodeArgs &a) {
    const auto &c = a.cache;
    const bool q8 = c.dtype == LRKV_FP8_E4M3;
    AnyParams P;
    P.q = a.q;
    P.S_K = c.S_K;
    P.S_V = c.S_V;
    P.R_K = c.R_K;
    P.R_V = c.R_V;
    P.B_K = a.B_K;
    P.B_V = a.B_V;
    P.N_K = c.N_K;
    P.out = a.out;
    P.seq_lens = a.seq_lens;
    P.page_table = a.page_table;
    P.req_row = a.req_row;
    P.max_pages = a.max_pages;
    P.num_pages = c.num_pages;
    P.page_size = c.page_size;
    P.max_len = decode_max_len(a);
    P.window = a.window;
    P.sinks = a.sinks;
    P.H = c.H;
    P.d_h = c.d_h;
    P.r = c.r;
    P.s_stride = cache_groups(c) * c.d_h;
    P.hpg = c.H / cache_groups(c);
    P.scale_log2 = 1.4426950408889634f / sqrtf((float)c.d_h);
    P.sc = q8 ? make_float4(c.scale[0], c.scale[1], c.scale[2], c.scale[3]) : make_float4(1.f, 1.f, 1.f, 1.f);
    P.status = a.status;
    // as many CTAs per (request, head) as leave every group four rows or more and
    // the GPU no more than about four CTAs per SM
    const int64_t rows = std::min<int64_t>(a.max_seq_len, (int64_t)a.window + a.sinks);
    int CL = 1;
    while (CL < 8 && rows >= (int64_t)8 * kGroups * CL && (int64_t)a.B * c.H * CL * 2 <= 4 * device_sm_count()) CL *= 2;
    if ((int64_t)a.B * CL > INT32_MAX) return cudaErrorInvalidValue;
    if (q8) return launch_sized<__nv_bfloat16, uint8_t, 1, 4>(P, a.B, CL, a.stream);
    if (c.dtype == LRKV_BF16) return launch_sized<__nv_bfloat16, __nv_bfloat16, 1, 4>(P, a.B, CL, a.stream);
    return launch_sized<float, float, 2, 8>(P, a.B, CL, a.stream);
}

}  // namespace lrkv
