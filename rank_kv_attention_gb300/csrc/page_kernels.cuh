// Internal interface between the C-ABI layer and the page-plan kernel.
#pragma once

#include "lrkv_common.cuh"

namespace lrkv {

struct PagePlanArgs {
    const int32_t *seq_lens, *new_rows;
    int B, max_pages, page_size, num_pages, window, sinks, max_rows;
    int32_t *page_table;
    const int32_t *free_pages, *n_free;
    int32_t *seq_lens_out, *cu_rows, *positions, *seq_ids, *slots, *free_out, *n_free_out;
    int32_t *status;
};
cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s);

int device_sm_count();  // SMs of the current device (lrkv_api.cu)

}  // namespace lrkv
