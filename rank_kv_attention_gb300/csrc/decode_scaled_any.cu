// Decode over the block-scaled cache (lrkv_decode_scaled) for any supported shape,
// and the merge of partial states that both of its kernels use.
//
//   x_j  = (2^eSK q.S_K[j] + 2^eRK[h] p.R_K[h,j]) / sqrt(d_h),   p = q B_K[h]
//   o    = sum_j a_j 2^eSV S_V[j] + (sum_j a_j 2^eRV[h] R_V[h,j]) B_V[h]^T,  a = softmax(x)
// (reading note "Low-Rank Key Value Attention", equations 6 and 7, on codes and
// scale exponents).  All in fp32.
//
// One CTA takes a part of a request's rows for one head.  A warp takes 32 rows at
// a time: lane j scores row j (q and p from shared memory), the warp updates its
// running maxima and sum, then its lanes add the rows' values up, four columns each,
// eight loads of a pool on their way at once.  A row's place and weights go to those lanes through
// shared memory: by shuffles the registers that hold them are missing for the loads.  The shared rows
// are read again by every head (out of L2), and the four warps' states meet in shared memory.
//
// Bound by the lanes' loads of rows r or d_h bytes apart, their latency, and the conversions of
// every code, once a head.  In a graph, 16 requests of 4096 rows: d_h = 64, r = 16, 8 heads
// 33 us (3.7 at the copy bandwidth); d_h = 32, r = 40, 6 heads 26; d_h = 128, r = 72, 12 heads 111
// (19.2); d_h = 128, r = 16, 40 heads 234 (14.9).  With places and weights by shuffles 38, 30, 140 and
// 310, and one load of a row's values at a time 86, 63, 240 and 605.
#include <algorithm>

#include "scaled_kernels.cuh"

namespace lrkv {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;

struct AnyArgs {
    ScaledDecodeArgs d;
    ScaledStates st;
    int splits;
    float scale_log2;
};

__device__ __forceinline__ void widen4(uint32_t w, float (&x)[4]) {
    const uint32_t a = f16x2_from_e4m3x2((uint16_t)w), b = f16x2_from_e4m3x2((uint16_t)(w >> 16));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    x[0] = f.x; x[1] = f.y; x[2] = g.x; x[3] = g.y;
}
// sum of eight codes times y
__device__ __forceinline__ float dot8(const uint2 &w, const float *y, float s) {
    float x[4];
    const float4 a = reinterpret_cast<const float4 *>(y)[0], b = reinterpret_cast<const float4 *>(y)[1];
    widen4(w.x, x);
    s = fmaf(x[0], a.x, s); s = fmaf(x[1], a.y, s); s = fmaf(x[2], a.z, s); s = fmaf(x[3], a.w, s);
    widen4(w.y, x);
    s = fmaf(x[0], b.x, s); s = fmaf(x[1], b.y, s); s = fmaf(x[2], b.z, s); s = fmaf(x[3], b.w, s);
    return s;
}

// NI: groups of 128 value columns.  HALF (64 columns at most): a half-warp adds a row's values up, so
// a warp takes two rows at a time, and the next rows' pages are looked up ahead in 72
// registers (with shuffles, 37 us of the first case above, 42 in 96, 47 without the look ahead; with
// 128 columns it cost registers that the loads need: 140 us of the third, 168 with it).
template <int NI, bool HALF>
__global__ void __launch_bounds__(kThreads, HALF ? 7 : 5) decode_scaled_any_kernel(const __grid_constant__ AnyArgs P) {
    constexpr int kRows = 8, kStep = HALF ? 2 : 1;  // loads on their way, rows of one
    __shared__ __align__(16) float qs[256], ps[256];
    __shared__ __align__(16) float tops[3][kWarps];  // m, ks, kr
    __shared__ float ls[kWarps], red[kWarps][512];
    // of the rows that a warp adds up: row of the pool, weights of the shared and the private value
    __shared__ int at[kWarps][32];
    __shared__ float2 weight[kWarps][32];
    const ScaledDecodeArgs &a = P.d;
    const ScaledPools &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / P.splits, sp = blockIdx.x % P.splits, h = blockIdx.y;
    const int d_h = c.d_h, r = c.r, H = c.H, g = h / (H / c.G);
    pdl_wait();
    pdl_launch_dependents();
    const int32_t L = a.seq_lens[b];
    const bool valid = L >= 1 && (int64_t)L <= (int64_t)a.max_pages * c.page_size;
    // rows of this part: a multiple of a CTA's step, so that parts are even
    const int part = valid ? ((L + P.splits - 1) / P.splits + kThreads - 1) / kThreads * kThreads : 0;
    const int64_t first = (int64_t)sp * part;
    const int begin = (int)min(first, (int64_t)(valid ? L : 0)), end = (int)min(first + part, (int64_t)(valid ? L : 0));

    const int64_t slot = (int64_t)b * P.splits + sp;
    float4 *head = P.st.head + slot * H + h;
    if (begin >= end) {  // (an empty part: a state without weight)
        if (tid == 0) *head = make_float4(-INFINITY, 0.f, -INFINITY, -INFINITY);
        return;
    }
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + ((size_t)b * H + h) * d_h;
    for (int d = tid; d < d_h; d += kThreads) qs[d] = __bfloat162float(q[d]);
    __syncthreads();
    const __nv_bfloat16 *B = static_cast<const __nv_bfloat16 *>(a.B_K) + (size_t)h * d_h * r;
    for (int k = tid; k < r; k += kThreads) {
        float s = 0.f;
#pragma unroll 8
        for (int d = 0; d < d_h; ++d) s = fmaf(qs[d], __bfloat162float(B[(size_t)d * r + k]), s);
        ps[k] = s;
    }
    __syncthreads();

    const int32_t *table = a.page_table + (size_t)(a.req_row ? a.req_row[b] : b) * a.max_pages;
    const int sw = c.G * d_h, rw = H * r;  // bytes of a token's shared and private row
    // largest x, x - m + eS and x - m + eR so far, what the sums are relative to
    float m = -INFINITY, ks = -INFINITY, kr = -INFINITY, l = 0.f, as[NI][4] = {}, ar[NI][4] = {};
    const int col0 = HALF ? 4 * (lane & 15) : 4 * lane, half = HALF ? lane >> 4 : 0;
    auto lookup = [&](int j) {
        int row = -1;
        if (j < end) {
            const int32_t page = table[j / c.page_size];
            if (page < 0 || page >= c.num_pages) status_or(a.status, LRKV_STATUS_BAD_PAGE);
            else row = page * c.page_size + j % c.page_size;
        }
        return row;
    };
    int next = HALF ? lookup(begin + 32 * warp + lane) : 0;
    for (int t0 = begin + 32 * warp; t0 < end; t0 += kThreads) {
        const int row = HALF ? next : lookup(t0 + lane);
        if (HALF) next = lookup(t0 + kThreads + lane);  // (on its way meanwhile)
        float x = -INFINITY, vs = 0.f, vr = 0.f;
        if (row >= 0) {
            const int64_t eb = row / c.block;
            const int e0 = c.exp[0][eb * c.G + g], e1 = c.exp[1][eb * c.G + g], e2 = c.exp[2][eb * H + h],
                      e3 = c.exp[3][eb * H + h];
            const uint8_t *sk = c.code[0] + (int64_t)row * sw + g * d_h, *rk = c.code[2] + (int64_t)row * rw + h * r;
            float s = 0.f, t = 0.f;
#pragma unroll 4
            for (int d = 0; d < d_h; d += 16) {
                const uint4 w = *reinterpret_cast<const uint4 *>(sk + d);
                s = dot8(make_uint2(w.x, w.y), qs + d, s);
                s = dot8(make_uint2(w.z, w.w), qs + d + 8, s);
            }
#pragma unroll 4
            for (int k = 0; k < r; k += 8) t = dot8(*reinterpret_cast<const uint2 *>(rk + k), ps + k, t);
            x = (s * exp2i(clamp_exp(e0)) + t * exp2i(clamp_exp(e2))) * P.scale_log2;
            vs = (float)clamp_exp(e1);
            vr = (float)clamp_exp(e3);
        }
        const float mn = fmaxf(m, warp_max(x)), down = m - ref_of(mn);
        x -= ref_of(mn);
        vs += x;
        vr += x;
        ks += down;
        kr += down;
        const float sn = fmaxf(ks, warp_max(vs)), rn = fmaxf(kr, warp_max(vr));
        l = l * ex2f(down) + ex2f(x);
        const float alpha = ex2f(ks - ref_of(sn)), beta = ex2f(kr - ref_of(rn));
        weight[warp][lane] = make_float2(ex2f(vs - ref_of(sn)), ex2f(vr - ref_of(rn)));
        at[warp][lane] = row;
        __syncwarp();
        m = mn;
        ks = sn;
        kr = rn;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                as[i][e] *= alpha;
                ar[i][e] *= beta;
            }
        // (rows past the part, or on no page, are zeros of weight zero)
#pragma unroll 1
        for (int t = 0; t < min(32, end - t0); t += kRows * kStep) {
            uint32_t cs[NI][kRows], cr[NI][kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int rt = at[warp][t + u * kStep + half];
                const uint8_t *sv = c.code[1] + (int64_t)rt * sw + g * d_h, *rv = c.code[3] + (int64_t)rt * rw + h * r;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int col = col0 + 128 * i;
                    cs[i][u] = rt >= 0 && col < d_h ? *reinterpret_cast<const uint32_t *>(sv + col) : 0;
                    cr[i][u] = rt >= 0 && col < r ? *reinterpret_cast<const uint32_t *>(rv + col) : 0;
                }
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const float2 w = weight[warp][t + u * kStep + half];
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    float y[4];
                    widen4(cs[i][u], y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) as[i][e] = fmaf(w.x, y[e], as[i][e]);
                    widen4(cr[i][u], y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) ar[i][e] = fmaf(w.y, y[e], ar[i][e]);
                }
            }
        }
        __syncwarp();
    }
    if (HALF)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            as[0][e] += __shfl_xor_sync(0xffffffffu, as[0][e], 16);
            ar[0][e] += __shfl_xor_sync(0xffffffffu, ar[0][e], 16);
        }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
        ls[warp] = l;
        tops[0][warp] = m;
        tops[1][warp] = ks;
        tops[2][warp] = kr;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int col = col0 + 128 * i;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (col < d_h) red[warp][col + e] = as[i][e];
            if (col < r) red[warp][256 + col + e] = ar[i][e];
        }
    }
    __syncthreads();
    // the four warps' sums: v of warp w, relative to its k-th maximum, relative to the largest of those
    auto most = [](const float4 &t) { return fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w)); };
    auto maxima = [&](int k) {
        const float4 t = *reinterpret_cast<const float4 *>(tops[0]);
        if (!k) return t;
        const float4 u = *reinterpret_cast<const float4 *>(tops[k]);
        const float m = ref_of(most(t));
        return make_float4(u.x + (t.x - m), u.y + (t.y - m), u.z + (t.z - m), u.w + (t.w - m));
    };
    auto join = [&](int k, const float *v, int step) {
        const float4 t = maxima(k);
        const float ref = ref_of(most(t));
        return (v[0] * ex2f(t.x - ref) + v[step] * ex2f(t.y - ref)) +
               (v[2 * step] * ex2f(t.z - ref) + v[3 * step] * ex2f(t.w - ref));
    };
    float *acc = P.st.acc + slot * H * (d_h + r);
#pragma unroll 1
    for (int i = tid; i < d_h + r; i += kThreads) {
        const bool priv = i >= d_h;
        const float s = join(priv ? 2 : 1, &red[0][priv ? 256 + i - d_h : i], 512);
        acc[priv ? (size_t)H * d_h + h * r + i - d_h : (size_t)h * d_h + i] = s;
    }
    if (tid == 0) *head = make_float4(most(maxima(0)), join(0, ls, 1), most(maxima(1)), most(maxima(2)));
}

// ---------------------------------------------------------------------------
// Merge: one CTA per (request, head).  With M the largest m_s, KS the largest m_s - M + kS_s (of all
// states), f_s = 2^(m_s - M), gS_s = 2^(m_s - M + kS_s - KS) and l = sum_s f_s l_s, the mean
// is S = 2^KS (sum_s gS_s accS_s) / l, that of the private rows R alike, and o = S + R B_V[h]^T.
// (KS and KR lie in the exponents' range.)  Groups of threads, one thread a column, take the states in
// turn.
//
// All of it is latency (about a microsecond for a round trip to memory that other
// SMs have just written): before the wait it reads what is there already, B_V[h] and the
// places of the request's states; after it everything else at once, value sums
// together with the maxima that weigh them.  HELD: value sums a thread has on the way.
// ---------------------------------------------------------------------------
constexpr int kMergeStates = 256, kMergeB = 3;

template <int THREADS, int HELD>
__global__ void __launch_bounds__(THREADS, HELD == 4 ? 6 : 2) scaled_merge_kernel(const __grid_constant__ ScaledMergeArgs P) {
    constexpr int kAhead = HELD == 4 ? 4 : 8;  // (four held: eight more would spill B_V)
    __shared__ float gs[2][kMergeStates], sums[512], part[kMergeB * THREADS];
    __shared__ float red[4][THREADS / 32], up[2];
    const int h = blockIdx.y, b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int H = P.H, d_h = P.d_h, r = P.r, W = d_h + r, cols = (W + 31) & ~31;
    // ---- B_V[h] in tasks of eight columns of a row: the first ones of every thread.  (The
    // kernel before this one started after all that is in front of the call was done.)
    const int v8 = r / 8, tasks = d_h * v8;
    const uint4 *B = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(P.B_V) + (size_t)h * d_h * r);
    uint4 bv[kMergeB];
#pragma unroll
    for (int j = 0; j < kMergeB; ++j)
        if (tid + j * THREADS < tasks) bv[j] = B[tid + j * THREADS];
    int2 place = P.places ? P.places[b] : make_int2(b * P.splits, P.splits);
    pdl_wait();
    pdl_launch_dependents();
    if (!P.places) {
        const int32_t L = P.seq_lens[b];
        if (L == -1 && P.leave) return;
        if (L < 1 || L > P.max_len) {
            // (of a prefill's rows the append and scaled_row_queries_kernel have said it)
            if (h == 0 && tid == 0 && !P.leave) status_or(P.status, LRKV_STATUS_BAD_SEQLEN);
            place.y = 0;
        }
    }
    const int ns = place.y;  // at most 256 parts, or a state of every CTA
    const int64_t s0 = place.x;
    float4 st = make_float4(-INFINITY, 0.f, -INFINITY, -INFINITY);
    const float4 *heads = P.st.head + (s0 * H + h);
    if (tid < ns) st = heads[tid * H];
    const int groups = max(1, THREADS / cols), g = tid / cols, c0 = tid - g * cols;
    const bool mine = g < groups && c0 < W;
    auto column = [&](int c) { return P.st.acc + s0 * H * W + (c < d_h ? h * d_h + c : H * d_h + h * r + c - d_h); };
    const float *acc = column(c0);
    float held[HELD];
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
        const int s = g + j * groups;
        held[j] = mine && s < ns ? acc[(int64_t)s * H * W] : 0.f;
    }
    // (the warps that hold states, most often one: then they need not meet before)
    const int nw = max(1, (ns + 31) / 32);
    float M = -INFINITY, KS = -INFINITY, KR = -INFINITY;  // (KS, KR: less M)
    if (warp < nw) {
        M = warp_max(st.x);
        st.z += st.x - ref_of(M);
        st.w += st.x - ref_of(M);
        KS = warp_max(st.z);
        KR = warp_max(st.w);
        if (lane == 0) {
            red[0][warp] = M;
            red[2][warp] = KS;
            red[3][warp] = KR;
        }
    }
    if (nw > 1) {
        __syncthreads();
        if (warp < nw) {
            const int w = lane < nw ? lane : 0;
            const float was = ref_of(M);
            M = warp_max(red[0][w]);
            KS = warp_max(red[2][w] + (red[0][w] - ref_of(M)));
            KR = warp_max(red[3][w] + (red[0][w] - ref_of(M)));
            st.z += was - ref_of(M);
            st.w += was - ref_of(M);
        }
    }
    if (warp < nw) {
        if (tid == 0) {
            up[0] = ex2f(KS);
            up[1] = ex2f(KR);
        }
        // a part without rows (m = -inf, l = 0) has written no value sums
        const bool none = st.x == -INFINITY && st.y == 0.f;
        gs[0][tid] = none ? -1.f : ex2f(st.z - ref_of(KS));
        gs[1][tid] = none ? -1.f : ex2f(st.w - ref_of(KR));
        float l = none ? 0.f : st.y * ex2f(st.x - ref_of(M));
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) red[1][warp] = l;
    }
    __syncthreads();
    float l = red[1][0];
#pragma unroll 1
    for (int w = 1; w < nw; ++w) l += red[1][w];
    const float inv = l != 0.f ? 1.f / l : 0.f;  // (NaN stays NaN)
    auto weigh = [&](int s, bool priv, float v) {
        const float k = gs[priv][s];
        return k >= 0.f || k != k ? k * v : 0.f;
    };
    const bool priv = c0 >= d_h;
    float x = 0.f;
    if (mine) {
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            if (g + j * groups < ns) x += weigh(g + j * groups, priv, held[j]);
#pragma unroll kAhead
        for (int s = g + HELD * groups; s < ns; s += groups) x += weigh(s, priv, acc[(int64_t)s * H * W]);
    }
    if (groups > 1) {
        sums[tid] = x;
        __syncthreads();
        if (g == 0 && c0 < W)
            for (int k = 1; k < groups; ++k) x += sums[k * cols + c0];
        __syncthreads();
    }
    // (by l first: a sum of many rows fits next to its own scale, not in the value's)
    if (g == 0 && c0 < W) sums[c0] = x * inv * up[priv];
    for (int c = tid + THREADS; c < W; c += THREADS) {  // (wider than the block)
        const float *a = column(c);
        x = 0.f;
        for (int s = 0; s < ns; ++s) x += weigh(s, c >= d_h, a[(int64_t)s * H * W]);
        sums[c] = x * inv * up[c >= d_h];
    }
    __syncthreads();
    // ---- expand
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(P.out) + ((size_t)b * H + h) * d_h;
    auto dot = [&](int task, const uint4 &w) {
        const float *o = sums + d_h + task % v8 * 8;
        float s = o[0] * bf16lo(w.x);
        s = fmaf(o[1], bf16hi(w.x), s); s = fmaf(o[2], bf16lo(w.y), s); s = fmaf(o[3], bf16hi(w.y), s);
        s = fmaf(o[4], bf16lo(w.z), s); s = fmaf(o[5], bf16hi(w.z), s); s = fmaf(o[6], bf16lo(w.w), s);
        return fmaf(o[7], bf16hi(w.w), s);
    };
    const bool fit = tasks <= kMergeB * THREADS;
    if (fit) {
#pragma unroll
        for (int j = 0; j < kMergeB; ++j)
            if (tid + j * THREADS < tasks) part[tid + j * THREADS] = dot(tid + j * THREADS, bv[j]);
        __syncthreads();
    }
    for (int d = tid; d < d_h; d += THREADS) {
        float s = sums[d];
        for (int k = 0; k < v8; ++k) s += fit ? part[d * v8 + k] : dot(k, B[d * v8 + k]);
        out[d] = __float2bfloat16_rn(s);
    }
}

__global__ void scaled_row_queries_kernel(const __grid_constant__ ScaledRows rows, int page_size, int max_len,
                                          int32_t *len, int32_t *req_row) {
    pdl_wait();
    pdl_launch_dependents();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= rows.n) return;
    const int b = request_of_row(rows.cu_rows, rows.B, i);
    if (b == rows.B || rows.cu_rows[b] > i) {
        len[i] = -1;
        req_row[i] = 0;
        return;
    }
    const int64_t pos = (int64_t)rows.start_pos[b] + (i - rows.cu_rows[b]);
    // (a row that has no place in the table was flagged as it was not written)
    if (pos >= max_len && pos < (int64_t)rows.max_pages * page_size) status_or(rows.status, LRKV_STATUS_BAD_SEQLEN);
    len[i] = pos >= 0 && pos < max_len ? (int)pos + 1 : 0;
    req_row[i] = b;
}

// Parts per request: enough CTAs for the device, of at least 128 rows each.
int any_splits(const ScaledPools &c, int B, int max_seq_len) {
    const int64_t most = ((int64_t)max_seq_len + kThreads - 1) / kThreads;
    const int64_t want = (8 * (int64_t)device_sm_count() + (int64_t)B * c.H - 1) / ((int64_t)B * c.H);
    return (int)std::max<int64_t>(1, std::min<int64_t>({most, want, 256}));
}

}  // namespace

size_t scaled_any_ws_bytes(const ScaledPools &c, int B, int max_seq_len) {
    // B * splits is at most 8 SMs / H + B, which grows with B, and at most 256 B
    const int64_t slots = std::min<int64_t>(8 * (int64_t)device_sm_count() / c.H + 1 + B,
                                            B * std::min<int64_t>(((int64_t)max_seq_len + kThreads - 1) / kThreads, 256));
    return scaled_states_bytes(slots, c.H, c.d_h, c.r);
}

cudaError_t launch_decode_scaled_any(const ScaledDecodeArgs &a, void *ws) {
    AnyArgs P;
    P.d = a;
    P.splits = any_splits(a.c, a.B, a.max_seq_len);
    P.st = scaled_states(ws, (int64_t)a.B * P.splits, a.c.H);
    P.scale_log2 = 1.4426950408889634f / sqrtf((float)a.c.d_h);
    const int cols = std::max(a.c.d_h, a.c.r);
    const auto kernel = cols <= 64    ? decode_scaled_any_kernel<1, true>
                        : cols <= 128 ? decode_scaled_any_kernel<1, false>
                                      : decode_scaled_any_kernel<2, false>;
    cudaError_t e = launch_pdl(kernel, dim3((unsigned)(a.B * P.splits), a.c.H), dim3(kThreads), 0, a.stream, P);
    if (e != cudaSuccess) return e;
    ScaledMergeArgs m;
    m.st = P.st;
    m.places = nullptr;
    m.splits = P.splits;
    m.seq_lens = a.seq_lens;
    m.max_len = a.max_pages * a.c.page_size;
    m.leave = a.req_row != nullptr;
    m.B_V = a.B_V;
    m.out = a.out;
    m.B = a.B;
    m.H = a.c.H;
    m.d_h = a.c.d_h;
    m.r = a.c.r;
    m.status = a.status;
    return launch_scaled_merge(m, a.stream);
}

cudaError_t launch_scaled_row_queries(const ScaledRows &rows, int page_size, int max_len, int32_t *len,
                                      int32_t *req_row, cudaStream_t s) {
    return launch_pdl(scaled_row_queries_kernel, dim3((rows.n + 255) / 256), dim3(256), 0, s, rows, page_size, max_len, len,
                      req_row);
}

cudaError_t launch_scaled_merge(const ScaledMergeArgs &m, cudaStream_t s) {
    // 512 threads with 16 value sums each on the way where CTAs are few, and states of a
    // request many (a decode of 4 requests of 32768 rows 65.6 us, 69.4 with 256 threads; of 1500
    // rows 16.3 and 17.2); else six CTAs of 256 threads an SM (of 64 ragged requests this kernel
    // took 12 us with 512, 9.5 so)
    const bool few = (int64_t)m.B * m.H < 2 * device_sm_count();
    return few ? launch_pdl(scaled_merge_kernel<512, 16>, dim3(m.B, m.H), dim3(512), 0, s, m)
               : launch_pdl(scaled_merge_kernel<256, 4>, dim3(m.B, m.H), dim3(256), 0, s, m);
}

}  // namespace lrkv
