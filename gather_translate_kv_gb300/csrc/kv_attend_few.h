// Attention of few rows a sequence (kv_attend_few.cu).
#pragma once

#include "kv_attn_launch.h"

namespace gtkv {

struct SplitRecord;

struct FewSplit {
  SplitRecord* rec;   // one per worker
  float* part;        // [worker][head of the worker][slot][rows * (D + 2)]
  int64_t n_workers;
  int32_t hw;         // KV heads of a worker, one warp each
  int32_t min_share;  // steps
  int32_t max_new;    // sequences with more new tokens are another kernel's
  int32_t blocks;
  int32_t join;
  int32_t q_wide;     // query rows start on 16 bytes
  int32_t out_wide;   // out starts on 4 bytes
};

// Shared-memory limits of the kernels on the current device (pool creation).
cudaError_t prepare_attend_few();
int64_t attend_few_workspace(int32_t H, int32_t D, int sm_count);
cudaError_t launch_attend_few(const DevPool& p, const Batch& b, const AttendArgs& a, bool e4m3, int32_t max_new,
                              void* workspace, int sm_count, cudaStream_t s);

}  // namespace gtkv
