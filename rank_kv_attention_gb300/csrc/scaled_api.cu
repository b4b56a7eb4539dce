// C-ABI entry points of the block-scaled cache: argument validation on the host,
// workspace layout, and dispatch to the kernels.  Nothing here allocates.
#include <algorithm>

#include "api_common.cuh"
#include "append_kernels.cuh"
#include "scaled_kernels.cuh"

namespace lrkv {

namespace {

constexpr int kMost = INT32_MAX / 2;

int check_scaled(const lrkv_scaled_t *c) {
    if (!c) return LRKV_E_INVALID_ARG;
    const int st = check_dims(c->H, c->d_h, c->r, LRKV_FP8_E4M3);
    if (st) return st;
    const void *p[] = {c->S_K, c->S_V, c->R_K, c->R_V, c->E_S_K, c->E_S_V, c->E_R_K, c->E_R_V};
    for (const void *x : p)
        if (!x || !aligned16(x)) return LRKV_E_INVALID_ARG;
    if (c->num_pages < 1 || c->page_size < 16 || c->page_size > 1024 || c->page_size % 16) return LRKV_E_SHAPE;
    if ((int64_t)c->num_pages * c->page_size > kMost) return LRKV_E_SHAPE;
    if (c->G < 0 || c->G > c->H || c->H % std::max(c->G, 1)) return LRKV_E_SHAPE;
    if (c->block < 16 || c->block % 16 || c->page_size % c->block) return LRKV_E_SHAPE;
    if (c->reserved) return LRKV_E_INVALID_ARG;
    return LRKV_OK;
}

ScaledPools pools_of(const lrkv_scaled_t &c) {
    ScaledPools p;
    void *code[4] = {c.S_K, c.S_V, c.R_K, c.R_V};
    uint8_t *exp[4] = {c.E_S_K, c.E_S_V, c.E_R_K, c.E_R_V};
    for (int k = 0; k < 4; ++k) {
        p.code[k] = static_cast<uint8_t *>(code[k]);
        p.exp[k] = exp[k];
    }
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.H = c.H;
    p.d_h = c.d_h;
    p.r = c.r;
    p.G = std::max(c.G, 1);
    p.block = c.block;
    return p;
}

// The requests' rows of a call (pointers unchecked where n is 0).
int check_rows(const lrkv_scaled_t *c, const int32_t *cu_rows, const int32_t *start_pos, int B, int n,
               const int32_t *page_table, int max_pages) {
    const int st = check_scaled(c);
    if (st) return st;
    if (n < 0 || n > kMost || B < 1 || max_pages < 1) return LRKV_E_SHAPE;
    if ((int64_t)max_pages * c->page_size > kMost) return LRKV_E_SHAPE;
    // blocks that n rows of B requests can lie in: one launch's grid
    if (n / c->block + 2 * (int64_t)B > kMost) return LRKV_E_SHAPE;
    if (n && (!cu_rows || !start_pos || !page_table)) return LRKV_E_INVALID_ARG;
    return LRKV_OK;
}

int check_strided(const lrkv_scaled_t *c, const void *const *x, const int64_t *ld, int dtype) {
    if (dtype != LRKV_F32 && dtype != LRKV_BF16) return LRKV_E_DTYPE;
    const int64_t per16 = dtype == LRKV_F32 ? 4 : 8;
    for (int k = 0; k < 4; ++k) {
        const int64_t row = k < 2 ? (int64_t)std::max(c->G, 1) * c->d_h : (int64_t)c->H * c->r;
        if (ld[k] < row || ld[k] % per16 || ld[k] > kMost) return LRKV_E_SHAPE;
        if (!x[k] || !aligned16(x[k])) return LRKV_E_INVALID_ARG;
    }
    return LRKV_OK;
}

// fp32 rows of the four pools, as the projection leaves them.
struct StagedRows {
    float *x[4];
    int64_t ld[4];
    size_t bytes;
};
StagedRows staged_rows(void *base, const ScaledPools &c, int n) {
    StagedRows s;
    size_t o = 0;
    for (int k = 0; k < 4; ++k) {
        s.ld[k] = (int64_t)c.heads(k) * c.width(k);
        s.x[k] = reinterpret_cast<float *>(static_cast<char *>(base) + o);
        o += align256(sizeof(float) * (size_t)n * s.ld[k]);
    }
    s.bytes = o;
    return s;
}

int check_projection(const void *X, int n, int d, const void *W_S_K, const void *W_S_V, const void *U_K,
                     const void *U_V, const lrkv_scaled_t *c) {
    if (d < 1 || d > 65536 || d % 8) return LRKV_E_SHAPE;
    if (!n) return LRKV_OK;
    const void *p[] = {X, W_S_K, W_S_V, U_K, U_V};
    for (const void *x : p)
        if (!x || !aligned16(x)) return LRKV_E_INVALID_ARG;
    // (a launch of the any-shape projection holds that many rows)
    if (n > 65535 * 32 && !tc_append_supported(n, d, std::max(c->G, 1) * c->d_h, c->H, c->r)) return LRKV_E_SHAPE;
    return LRKV_OK;
}

cudaError_t run_append_scaled(const void *X, const ScaledRows &rows, int d, const void *W_S_K, const void *W_S_V,
                              const void *U_K, const void *U_V, const ScaledPools &c, const StagedRows &st,
                              cudaStream_t s, void *const *y = nullptr, int ypages = 0) {
    if (append_scaled_tc_fits(c, rows.n, rows.B, d)) {
        ScaledAppendArgs p = {c, rows, X, W_S_K, W_S_V, U_K, U_V, d, {nullptr, nullptr, nullptr, nullptr}, ypages, s};
        for (int k = 0; y && k < 4; ++k) p.y[k] = y[k];
        prof_before(LRKV_PROFILE_PROJECTION, s);
        const cudaError_t e = launch_append_scaled_tc(p);
        prof_after(LRKV_PROFILE_PROJECTION, s);
        return e;
    }
    AppendArgsT<__nv_bfloat16> a = {};
    a.X = static_cast<const __nv_bfloat16 *>(X);
    a.n = rows.n;
    a.d = d;
    a.W_S_K = static_cast<const __nv_bfloat16 *>(W_S_K);
    a.W_S_V = static_cast<const __nv_bfloat16 *>(W_S_V);
    a.U_K = static_cast<const __nv_bfloat16 *>(U_K);
    a.U_V = static_cast<const __nv_bfloat16 *>(U_V);
    a.B = rows.B;
    a.H = c.H;
    a.d_h = c.G * c.d_h;
    a.r = c.r;
    a.page_size = c.page_size;
    a.status = rows.status;
    a.stream = s;
    ScaledWriteArgs w;
    for (int k = 0; k < 4; ++k) {
        a.rows32[k] = st.x[k];
        w.x[k] = st.x[k];
        w.ld[k] = st.ld[k];
    }
    prof_before(LRKV_PROFILE_PROJECTION, s);
    cudaError_t e = dispatch_append(a);
    prof_after(LRKV_PROFILE_PROJECTION, s);
    if (e != cudaSuccess) return e;
    w.c = c;
    w.rows = rows;
    w.f32 = true;
    w.stream = s;
    return launch_write_scaled(w);
}

int run_decode_scaled(const ScaledDecodeArgs &a, void *ws) {
    prof_before(LRKV_PROFILE_ATTENTION, a.stream);
    const bool tc = !a.req_row && scaled_tc_covers(a.c);
    const cudaError_t e = tc ? launch_decode_scaled_tc(a, ws) : launch_decode_scaled_any(a, ws);
    prof_after(LRKV_PROFILE_ATTENTION, a.stream);
    return e == cudaSuccess ? LRKV_OK : cuda_fail(e);
}

size_t decode_scaled_ws_bytes(const ScaledPools &c, int B, int max_seq_len) {
    return scaled_tc_covers(c) ? scaled_tc_ws_bytes(c, B, max_seq_len) : scaled_any_ws_bytes(c, B, max_seq_len);
}

// Prefill workspace: the projected rows, and over them, when those have been written, tiled, the
// bf16 pools of the values with their page table, or, a decode a row, the rows' places and the
// decode's workspace.  (The append in one kernel has no projected rows, and lays values out.)
struct PrefillScaledWs {
    StagedRows rows;
    bool tiled, own_pages;
    lrkv_cache_t cache;  // tiled
    int32_t *table;
    int pages;
    int32_t *len, *req_row;
    void *dec;
    size_t bytes;
};
bool prefill_scaled_tiles(const lrkv_scaled_t &c, int B, int n, int max_ctx) {
    // (requests and query tiles are a grid's y and z; the layout's CTAs of 4 or 8 rows its x)
    return c.d_h == 128 && c.G <= 1 && c.r <= 64 && c.page_size % 64 == 0 && B <= 65535 &&
           std::min(n, max_ctx) <= 65535 * 128 && B * (((int64_t)max_ctx + 7) / 8) <= INT32_MAX;
}
PrefillScaledWs prefill_scaled_ws(void *base, const lrkv_scaled_t &sc, int B, int n, int max_ctx) {
    const ScaledPools c = pools_of(sc);
    PrefillScaledWs w = {};
    w.rows = staged_rows(base, c, n);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        void *p = static_cast<char *>(base) + o;
        o += align256(bytes);
        return p;
    };
    w.pages = (int)(((int64_t)max_ctx + 63) / 64);
    // pages of the requests' own, or, where the whole pool is smaller, its pages
    const int64_t own = (int64_t)B * w.pages * 64, all = (int64_t)c.num_pages * c.page_size;
    w.own_pages = own <= all;
    const int64_t rows = std::min(own, all);
    w.tiled = prefill_scaled_tiles(sc, B, n, max_ctx) && rows + 64 < INT32_MAX / 2;
    if (w.tiled) {
        w.cache = lrkv_cache_t{};
        w.cache.S_K = take(2 * (size_t)rows * c.d_h);
        w.cache.S_V = take(2 * (size_t)rows * c.d_h);
        w.cache.R_K = take(2 * (size_t)rows * c.H * c.r);
        w.cache.R_V = take(2 * (size_t)rows * c.H * c.r);
        w.cache.page_size = w.own_pages ? 64 : c.page_size;
        w.cache.num_pages = (int32_t)(rows / w.cache.page_size);
        w.cache.H = c.H;
        w.cache.d_h = c.d_h;
        w.cache.r = c.r;
        w.cache.dtype = LRKV_BF16;
        w.cache.G = 1;
        if (w.own_pages) w.table = static_cast<int32_t *>(take(sizeof(int32_t) * (size_t)B * w.pages));
    } else {
        const size_t arr = sizeof(int32_t) * (size_t)n;
        w.len = static_cast<int32_t *>(take(arr));
        w.req_row = static_cast<int32_t *>(take(arr));
        w.dec = take(scaled_any_ws_bytes(c, n, max_ctx));
    }
    w.bytes = std::max(o, w.rows.bytes);
    return w;
}

}  // namespace

}  // namespace lrkv

using namespace lrkv;

extern "C" {

int lrkv_write_scaled(const void *S_K, int64_t ld_sk, const void *S_V, int64_t ld_sv, const void *R_K, int64_t ld_rk,
                      const void *R_V, int64_t ld_rv, int32_t dtype, const int32_t *cu_rows, const int32_t *start_pos,
                      int32_t B, int32_t n, const lrkv_scaled_t *cache, const int32_t *page_table, int32_t max_pages,
                      int32_t *dev_status, lrkv_stream_t stream) {
    int st = check_rows(cache, cu_rows, start_pos, B, n, page_table, max_pages);
    if (st) return st;
    ScaledWriteArgs a;
    const void *x[4] = {S_K, S_V, R_K, R_V};
    const int64_t ld[4] = {ld_sk, ld_sv, ld_rk, ld_rv};
    if (n == 0) return dtype == LRKV_F32 || dtype == LRKV_BF16 ? LRKV_OK : LRKV_E_DTYPE;
    if ((st = check_strided(cache, x, ld, dtype))) return st;
    for (int k = 0; k < 4; ++k) {
        a.x[k] = x[k];
        a.ld[k] = ld[k];
    }
    a.c = pools_of(*cache);
    a.rows = {cu_rows, start_pos, B, n, page_table, max_pages, dev_status};
    a.f32 = dtype == LRKV_F32;
    a.stream = (cudaStream_t)stream;
    const cudaError_t e = launch_write_scaled(a);
    return e == cudaSuccess ? LRKV_OK : cuda_fail(e);
}

int lrkv_read_scaled(const lrkv_scaled_t *cache, const int32_t *cu_rows, const int32_t *start_pos, int32_t B, int32_t n,
                     const int32_t *page_table, int32_t max_pages, int32_t dtype, void *S_K, int64_t ld_sk, void *S_V,
                     int64_t ld_sv, void *R_K, int64_t ld_rk, void *R_V, int64_t ld_rv, int32_t *dev_status,
                     lrkv_stream_t stream) {
    int st = check_rows(cache, cu_rows, start_pos, B, n, page_table, max_pages);
    if (st) return st;
    ScaledReadArgs a;
    void *y[4] = {S_K, S_V, R_K, R_V};
    const int64_t ld[4] = {ld_sk, ld_sv, ld_rk, ld_rv};
    if (n == 0) return dtype == LRKV_F32 || dtype == LRKV_BF16 ? LRKV_OK : LRKV_E_DTYPE;
    if ((st = check_strided(cache, y, ld, dtype))) return st;
    for (int k = 0; k < 4; ++k) {
        a.y[k] = y[k];
        a.ld[k] = ld[k];
    }
    a.c = pools_of(*cache);
    a.rows = {cu_rows, start_pos, B, n, page_table, max_pages, dev_status};
    a.f32 = dtype == LRKV_F32;
    a.stream = (cudaStream_t)stream;
    const cudaError_t e = launch_read_scaled(a);
    return e == cudaSuccess ? LRKV_OK : cuda_fail(e);
}

size_t lrkv_append_scaled_workspace_bytes(const lrkv_scaled_t *cache, int32_t n) {
    if (check_scaled(cache) || n < 0) return 0;
    return staged_rows(nullptr, pools_of(*cache), n).bytes;
}

int lrkv_append_scaled(const void *X, const int32_t *cu_rows, const int32_t *start_pos, int32_t B, int32_t n, int32_t d,
                       const void *W_S_K, const void *W_S_V, const void *U_K, const void *U_V,
                       const lrkv_scaled_t *cache, const int32_t *page_table, int32_t max_pages, void *workspace,
                       size_t workspace_bytes, int32_t *dev_status, lrkv_stream_t stream) {
    int st = check_rows(cache, cu_rows, start_pos, B, n, page_table, max_pages);
    if (st || (st = check_projection(X, n, d, W_S_K, W_S_V, U_K, U_V, cache))) return st;
    if (n == 0) return LRKV_OK;
    const ScaledPools c = pools_of(*cache);
    const StagedRows rows = staged_rows(workspace, c, n);
    if (!workspace || !aligned256(workspace) || workspace_bytes < rows.bytes) return LRKV_E_WORKSPACE;
    const cudaError_t e = run_append_scaled(X, {cu_rows, start_pos, B, n, page_table, max_pages, dev_status}, d, W_S_K,
                                            W_S_V, U_K, U_V, c, rows, (cudaStream_t)stream);
    return e == cudaSuccess ? LRKV_OK : cuda_fail(e);
}

size_t lrkv_decode_scaled_workspace_bytes(const lrkv_scaled_t *cache, int32_t B, int32_t max_seq_len) {
    if (check_scaled(cache) || B < 1 || max_seq_len < 1) return 0;
    return decode_scaled_ws_bytes(pools_of(*cache), B, max_seq_len);
}

int lrkv_decode_scaled(const void *q, const lrkv_scaled_t *cache, const void *B_K, const void *B_V,
                       const int32_t *seq_lens, const int32_t *page_table, int32_t B, int32_t max_pages,
                       int32_t max_seq_len, void *out, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                       lrkv_stream_t stream) {
    const int st = check_scaled(cache);
    if (st) return st;
    if (B < 1 || max_pages < 1 || max_seq_len < 1) return LRKV_E_SHAPE;
    if ((int64_t)max_pages * cache->page_size > kMost) return LRKV_E_SHAPE;
    if ((int64_t)max_seq_len > (int64_t)max_pages * cache->page_size) return LRKV_E_BOUNDS;
    // lengths count up to the page table's end, whatever max_seq_len says: 2^24 units of 64
    // rows, whose products with a grid's size stay within 32 bits
    if ((int64_t)B * (((int64_t)max_pages * cache->page_size + 63) / 64) > (1 << 24)) return LRKV_E_SHAPE;
    const void *p[] = {q, B_K, B_V, out};
    for (const void *x : p)
        if (!x || !aligned16(x)) return LRKV_E_INVALID_ARG;
    if (!seq_lens || !page_table) return LRKV_E_INVALID_ARG;
    ScaledDecodeArgs a;
    a.c = pools_of(*cache);
    if (!workspace || !aligned256(workspace) || workspace_bytes < decode_scaled_ws_bytes(a.c, B, max_seq_len))
        return LRKV_E_WORKSPACE;
    a.q = q;
    a.B_K = B_K;
    a.B_V = B_V;
    a.seq_lens = seq_lens;
    a.page_table = page_table;
    a.req_row = nullptr;
    a.B = B;
    a.max_pages = max_pages;
    a.max_seq_len = max_seq_len;
    a.out = out;
    a.status = dev_status;
    a.stream = (cudaStream_t)stream;
    return run_decode_scaled(a, workspace);
}

size_t lrkv_prefill_scaled_workspace_bytes(const lrkv_scaled_t *cache, int32_t B, int32_t n, int32_t max_ctx) {
    if (check_scaled(cache) || B < 1 || n < 0 || max_ctx < 1) return 0;
    return prefill_scaled_ws(nullptr, *cache, B, n, max_ctx).bytes;
}

int lrkv_prefill_scaled(const void *X, const void *Q, const int32_t *cu_rows, const int32_t *start_pos, int32_t B,
                        int32_t n, int32_t max_ctx, int32_t d, const void *W_S_K, const void *W_S_V, const void *U_K,
                        const void *U_V, const void *B_K, const void *B_V, const lrkv_scaled_t *cache,
                        const int32_t *page_table, int32_t max_pages, void *out, void *workspace,
                        size_t workspace_bytes, int32_t *dev_status, lrkv_stream_t stream) {
    int st = check_rows(cache, cu_rows, start_pos, B, n, page_table, max_pages);
    if (st || (st = check_projection(X, n, d, W_S_K, W_S_V, U_K, U_V, cache))) return st;
    if (max_ctx < 1) return LRKV_E_SHAPE;
    if ((int64_t)max_ctx > (int64_t)max_pages * cache->page_size) return LRKV_E_BOUNDS;
    if (n == 0) return LRKV_OK;
    const void *ptrs[] = {Q, B_K, B_V, out};
    for (const void *x : ptrs)
        if (!x || !aligned16(x)) return LRKV_E_INVALID_ARG;
    const PrefillScaledWs w = prefill_scaled_ws(workspace, *cache, B, n, max_ctx);
    if (!workspace || !aligned256(workspace) || workspace_bytes < w.bytes) return LRKV_E_WORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    const ScaledPools c = pools_of(*cache);
    const ScaledRows rows = {cu_rows, start_pos, B, n, page_table, max_pages, dev_status};
    PrefillTcArgs p;
    if (w.tiled) {
        p.Q = Q;
        p.cu_rows = cu_rows;
        p.start_pos = start_pos;
        p.B = B;
        p.n = n;
        p.max_ctx = max_ctx;
        p.max_len = max_ctx;  // (values are laid out up to there)
        p.B_K = B_K;
        p.B_V = B_V;
        p.cache = w.cache;
        p.page_table = w.own_pages ? w.table : page_table;
        p.max_pages = w.own_pages ? w.pages : max_pages;
        p.out = out;
        p.status = dev_status;
        p.stream = s;
        p.split = p.early = true;  // (behind launch_expand_scaled, which lets it start after its own wait)
        if (!prefill_tc_fits(p)) return LRKV_E_SHAPE;  // (no tensor maps: their encoder is not there)
    }
    // (the append in one kernel lays its own rows' values out)
    void *const y[4] = {w.cache.S_K, w.cache.S_V, w.cache.R_K, w.cache.R_V};
    cudaError_t e = run_append_scaled(X, rows, d, W_S_K, W_S_V, U_K, U_V, c, w.rows, s, w.tiled ? y : nullptr,
                                      w.own_pages ? w.pages : 0);
    if (e != cudaSuccess) return cuda_fail(e);
    if (w.tiled) {
        ScaledExpandArgs x;
        x.c = c;
        x.rows = rows;
        for (int k = 0; k < 4; ++k) x.y[k] = y[k];
        x.history = append_scaled_tc_fits(c, n, B, d);
        x.table = w.table;
        x.pages = w.pages;
        x.max_ctx = max_ctx;
        x.stream = s;
        if ((e = launch_expand_scaled(x)) != cudaSuccess) return cuda_fail(e);
        prof_before(LRKV_PROFILE_ATTENTION, s);
        const int rc = launch_prefill_tc(p);
        prof_after(LRKV_PROFILE_ATTENTION, s);
        return rc == 0 ? LRKV_OK : cuda_fail(rc < 0 ? (cudaError_t)(-rc) : cudaErrorInvalidValue);
    }
    e = launch_scaled_row_queries(rows, c.page_size, max_ctx, w.len, w.req_row, s);
    if (e != cudaSuccess) return cuda_fail(e);
    ScaledDecodeArgs a;
    a.c = c;
    a.q = Q;
    a.B_K = B_K;
    a.B_V = B_V;
    a.seq_lens = w.len;
    a.page_table = page_table;
    a.req_row = w.req_row;
    a.B = n;
    a.max_pages = max_pages;
    a.max_seq_len = max_ctx;
    a.out = out;
    a.status = dev_status;
    a.stream = s;
    return run_decode_scaled(a, w.dec);
}

}  // extern "C"
