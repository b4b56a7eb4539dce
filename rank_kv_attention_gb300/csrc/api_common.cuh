// Shared by the files that hold C-ABI entry points.
#pragma once

#include "lrkv_common.cuh"

namespace lrkv {

// Remembers the error for lrkv_last_cuda_error; LRKV_E_CUDA.
int cuda_fail(cudaError_t e);
// Event pair around the dominant kernel of a call (kind: LRKV_PROFILE_*).
void prof_before(int kind, cudaStream_t s);
void prof_after(int kind, cudaStream_t s);
// Whether head count, widths and element type are supported (LRKV_OK or an error).
int check_dims(int H, int d_h, int r, int dtype);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

}  // namespace lrkv
