// Internal interface between the C-ABI layer and the kernels of the block-scaled
// cache (lrkv_scaled_t).
#pragma once

#include "lrkv_common.cuh"

namespace lrkv {

// Pools in the order S_K, S_V, R_K, R_V.
struct ScaledPools {
    uint8_t *code[4];
    uint8_t *exp[4];
    int num_pages, page_size, H, d_h, r, G, block;
    __host__ __device__ int heads(int k) const { return k < 2 ? G : H; }
    __host__ __device__ int width(int k) const { return k < 2 ? d_h : r; }
};

// Requests' rows of a call and where they lie.
struct ScaledRows {
    const int32_t *cu_rows, *start_pos;
    int B, n;
    const int32_t *page_table;
    int max_pages;
    int32_t *status;
};

struct ScaledWriteArgs {
    ScaledPools c;
    ScaledRows rows;
    const void *x[4];
    int64_t ld[4];
    bool f32;
    cudaStream_t stream;
};
cudaError_t launch_write_scaled(const ScaledWriteArgs &a);

struct ScaledReadArgs {
    ScaledPools c;
    ScaledRows rows;
    void *y[4];
    int64_t ld[4];
    bool f32;
    cudaStream_t stream;
};
cudaError_t launch_read_scaled(const ScaledReadArgs &a);

// Lays the cache rows 0 .. start_pos[b] + rows of b - 1 of every request out in
// bf16 pools y (dense rows) under a page size of 64: at pages of their own, b *
// pages + k, entered in `table` [B, pages], or (table NULL) at the pool rows they
// have in the cache.  The cache's page size is a multiple of 64.
struct ScaledExpandArgs {
    ScaledPools c;
    ScaledRows rows;
    void *y[4];
    int32_t *table;
    int pages;    // of 64 rows, a request
    int max_ctx;  // rows of a request that can be asked for
    bool history;  // only rows 0 .. start_pos[b] - 1 (the others are there)
    cudaStream_t stream;
};
cudaError_t launch_expand_scaled(const ScaledExpandArgs &a);

// What a one-query decode of every row of a call needs: its length (0: no valid position; -1: no request owns the row) and
// page-table row.
cudaError_t launch_scaled_row_queries(const ScaledRows &rows, int page_size, int max_len, int32_t *len,
                                      int32_t *req_row, cudaStream_t s);

struct ScaledDecodeArgs {
    ScaledPools c;
    const void *q, *B_K, *B_V;
    const int32_t *seq_lens, *page_table;
    const int32_t *req_row;  // page-table row of request b, or NULL: b.  Set: outputs of length -1 are left alone
    int B, max_pages, max_seq_len;
    void *out;
    int32_t *status;
    cudaStream_t stream;
};

// Partial softmax states of decode_scaled (log2 units): slot s holds, for every head, the
// running maximum m of the scores x and the sum of 2^(x - m), and the sums of 2^(x - m + e - k)
// code over shared and private rows, each relative to its own maximum k of x - m + e.  A value
// may be 2^128 or 2^-126 as it lies in the cache, and a sum of many such, or one that shares a
// factor with a weight below one, would leave fp32; these neither overflow nor vanish.  (The
// exponent is added to a score's distance from the largest: next to a large score it would
// lose its digits.)
struct ScaledStates {
    float4 *head;  // [slots][H]: m, sum, k of the shared rows, k of the private rows
    float *acc;    // [slots][H d_h | H r]
};
__host__ __device__ inline size_t scaled_states_bytes(int64_t slots, int H, int d_h, int r) {
    return align256(sizeof(float4) * (size_t)slots * H) + sizeof(float) * (size_t)slots * H * (d_h + r);
}
inline ScaledStates scaled_states(void *base, int64_t slots, int H) {
    return {static_cast<float4 *>(base),
            reinterpret_cast<float *>(static_cast<char *>(base) + align256(sizeof(float4) * (size_t)slots * H))};
}

// Any shape: one CTA per (request, split, head).  Workspace bytes of a call and
// of every smaller one.
size_t scaled_any_ws_bytes(const ScaledPools &c, int B, int max_seq_len);
cudaError_t launch_decode_scaled_any(const ScaledDecodeArgs &a, void *ws);

// On tensor cores: covered shapes (d_h = 128, one shared basis, H a multiple of 4 up
// to 32, r up to 64, operands that fit), workspace bytes and launcher (req_row NULL).
bool scaled_tc_covers(const ScaledPools &c);
size_t scaled_tc_ws_bytes(const ScaledPools &c, int B, int max_seq_len);
cudaError_t launch_decode_scaled_tc(const ScaledDecodeArgs &a, void *ws);

// Merges the states of every request and head into out.
struct ScaledMergeArgs {
    ScaledStates st;
    // first slot and count of request b's states, written before the kernel in front of
    // the merge lets it start, or NULL:
    const int2 *places;
    int splits;  // slots b * splits .. of every request whose length is valid
    const int32_t *seq_lens;
    int max_len;
    bool leave;  // outputs of length -1 are left alone
    const void *B_V;
    void *out;
    int B, H, d_h, r;
    int32_t *status;
};
cudaError_t launch_scaled_merge(const ScaledMergeArgs &m, cudaStream_t s);

int device_sm_count();  // SMs of the current device (lrkv_api.cu)

// Projection and write in one kernel, on tensor cores: covered shapes and launcher.  y:
// bf16 pools that get the values too (NULL: none), at row b * ypages * 64 + position, or
// (ypages 0) at the cache's row.
struct ScaledAppendArgs {
    ScaledPools c;
    ScaledRows rows;
    const void *X, *W_S_K, *W_S_V, *U_K, *U_V;
    int d;
    void *y[4];
    int ypages;
    cudaStream_t stream;
};
bool append_scaled_tc_fits(const ScaledPools &c, int n, int B, int d);
cudaError_t launch_append_scaled_tc(const ScaledAppendArgs &p);

// 2^x, flushing.  (Of -infinity 0.)
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Largest of a warp's values; NaN does not count.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// A maximum as the point that exponents are relative to: none of -infinity.
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

// Scale exponents.
__device__ __forceinline__ int clamp_exp(int byte) {
    return min(max(byte - 127, LRKV_SCALED_MIN_EXP), LRKV_SCALED_MAX_EXP);
}
// Least exponent e with |x| <= 448 * 2^e (448 = 1.75 * 2^8), in [LRKV_SCALED_MIN_EXP, most];
// x >= 0 finite (of the largest x it is 120).
__device__ __forceinline__ int needed_exp(float x, int most = LRKV_SCALED_MAX_EXP) {
    const uint32_t u = __float_as_uint(x);
    const int e = (int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, LRKV_SCALED_MIN_EXP), most);
}

// Four codes times s, rounded to codes again.
__device__ __forceinline__ uint32_t shrink_codes(uint32_t w, float s) {
    uint32_t r = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t h2 = f16x2_from_e4m3x2((uint16_t)(w >> (16 * k)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
        r |= (uint32_t)e4m3x2_from_f32(f.x * s, f.y * s) << (16 * k);
    }
    return r;
}

}  // namespace lrkv
