// Launchers of the operators that surround the layers (called by loop_api.cu after validation).
#pragma once

#include "../../include/dsv4_loop.h"
#include "dsv4_common.cuh"
#include "dsv4_launch.h"

namespace dsv4 {

cudaError_t launch_rope(const dsv4_rope_params& p, cudaStream_t s);
cudaError_t launch_rope_table(const dsv4_rope_table_params& p, cudaStream_t s);
cudaError_t launch_batch_plan(const dsv4_batch_plan_params& p, cudaStream_t s);
cudaError_t launch_draft_verify(const dsv4_draft_verify_params& p, cudaStream_t s);
cudaError_t read_flags_loop_plan(uint32_t* f);
cudaError_t read_flags_loop_verify(uint32_t* f);

}  // namespace dsv4
