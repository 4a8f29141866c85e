// The attention kernels behind launch_attend: few rows a sequence
// (kv_attend_few.cu) and tiles of rows (kv_attend_tile.cu), head sizes 64 and 128.
#pragma once

#include "kv_attn_launch.h"

namespace gtkv {

// Shared-memory limits of the kernels on the current device (pool creation).
cudaError_t prepare_attend_few();
cudaError_t prepare_attend_tile();
int64_t attend_few_workspace(int32_t H, int32_t D, int sm_count);
int64_t attend_tile_workspace(int32_t D, int sm_count);
// Sequences of at most max_new, and of at least min_new, new tokens.
cudaError_t launch_attend_few(const DevPool& p, const Batch& b, const AttendArgs& a, bool e4m3, int32_t max_new,
                              void* workspace, int sm_count, cudaStream_t s);
cudaError_t launch_attend_tile(const DevPool& p, const Batch& b, const AttendArgs& a, bool e4m3, int32_t min_new,
                               void* workspace, int sm_count, cudaStream_t s);

}  // namespace gtkv
