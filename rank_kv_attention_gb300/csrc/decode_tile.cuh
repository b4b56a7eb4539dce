// What the tensor-core decode kernels share: fragment helpers, the list of
// shapes, and the host's tensor maps (decode_fast.cu).
#pragma once

#include "decode_kernels.cuh"
#include "tc_common.cuh"

namespace lrkv {

__device__ __forceinline__ uint32_t ld_u32(const __nv_bfloat16 *p) {
    return *reinterpret_cast<const uint32_t *>(p);
}

// The running maximum (log2 units) only moves when a tile exceeds it by this
// much; weights stay below 2^kLazyMax, far inside fp32 range.
constexpr float kLazyMax = 8.f;

// Byte offset, inside a region of 64-column swizzled boxes of TS rows, of the
// 16-byte chunk `cc` (counted along the row) of row `j`.
template <int TS>
__device__ __forceinline__ uint32_t box_chunk_rows(int j, int cc) {
    return (uint32_t)((cc >> 3) * (TS * 128)) + swz128(j, cc & 7);
}

// 8-bit (E4M3) tiles: 32- and 16-bit words of codes, widened to f16 pairs
// (exact).
__device__ __forceinline__ uint32_t lds_u32(const uint8_t *p) {
    return *reinterpret_cast<const uint32_t *>(p);
}
__device__ __forceinline__ uint32_t lds_u16(const uint8_t *p) {
    return *reinterpret_cast<const uint16_t *>(p);
}
__device__ __forceinline__ uint32_t f16x2_lo(uint32_t w) { return f16x2_from_e4m3x2((uint16_t)w); }
__device__ __forceinline__ uint32_t f16x2_hi(uint32_t w) {
    return f16x2_from_e4m3x2((uint16_t)(w >> 16));
}

// A fragments of two value m-tiles from the 32-bit words of rows 2tq, 2tq+1,
// 2tq+8, 2tq+9 (the layout of 8-bit tiles is described in decode_fast.cu); MASK: zero invalid rows.
template <bool MASK>
__device__ __forceinline__ void q8_pair_frags(uint32_t w0, uint32_t w1, uint32_t w8, uint32_t w9,
                                              uint32_t m01, uint32_t m89, uint32_t (&a)[4],
                                              uint32_t (&b)[4]) {
    const uint32_t x01 = prmt<0x5140>(w0, w1), y01 = prmt<0x7362>(w0, w1);
    const uint32_t x89 = prmt<0x5140>(w8, w9), y89 = prmt<0x7362>(w8, w9);
    a[0] = f16x2_lo(x01); a[1] = f16x2_hi(x01); a[2] = f16x2_lo(x89); a[3] = f16x2_hi(x89);
    b[0] = f16x2_lo(y01); b[1] = f16x2_hi(y01); b[2] = f16x2_lo(y89); b[3] = f16x2_hi(y89);
    if (MASK) {
        a[0] &= m01; a[1] &= m01; a[2] &= m89; a[3] &= m89;
        b[0] &= m01; b[1] &= m01; b[2] &= m89; b[3] &= m89;
    }
}

// Value column (relative to the tile's or the warp's first column) of
// accumulator m-tile mt, element e, under the permutation of q8_values.
template <int KSP>
__device__ __forceinline__ int q8_value_col(int mt, int e, int gq) {
    return (mt < (KSP & ~1)) ? 32 * (mt >> 1) + 4 * gq + 2 * (mt & 1) + (e >> 1)
                             : 16 * mt + 2 * gq + (e >> 1);
}

// Map over a pool viewed as [rows, cols] elements of eb bytes (bf16, f16 or
// 8-bit codes), as three dimensions (128 / eb columns, rows, cols * eb / 128
// blocks of 128 bytes) with strides (eb, cols * eb, 128 bytes).  A box of
// (128 / eb) x 16 x box_blocks (default: all blocks) with 128-byte swizzle
// lands a 16-row tile as consecutive 16-row x 128-byte boxes (matches
// box_chunk).
bool make_map(CUtensorMap *map, const void *pool, int64_t rows, int cols, int eb, int box_blocks = 0,
              bool f16 = false, int box_rows = 16);

// Map over a row-major [rows, H] array of elements of eb bytes (bf16 joint
// key norms, fp32 given scores) as (H, rows, 1): a box of H x 16 x 1 lands a
// tile's 16 rows, unswizzled.
bool make_row_map(CUtensorMap *map, const void *base, int64_t rows, int H, int eb, int box_rows = 16);

// Shapes (H, r) of the tensor-core decode (bf16 and 8-bit caches, d_h = 128).
#define LRKV_FAST_SHAPES(X) X(16, 16) X(16, 32) X(16, 48) X(16, 56) X(16, 64) X(32, 16) X(32, 32)

// Shapes the tensor-core decode serves with two shared groups (bf16).
#define LRKV_FAST_SHAPES_G2(X) X(16, 32) X(16, 48)

}  // namespace lrkv
