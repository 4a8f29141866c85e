// Host launchers of the operators of kv_attention.h; each enqueues on `s` and
// returns the launch status.
#pragma once

#include "kv_attention.h"
#include "kv_batch.cuh"

namespace gtkv {

cudaError_t launch_append(const DevPool& p, const Batch& b, int32_t layer, int32_t type, bool e4m3, int32_t H,
                          int32_t D, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const kv_rotary* rot, const void* q, int64_t q_stride, int32_t Q, void* q_out, float* scales,
                          int sm_count, cudaStream_t s);

cudaError_t launch_gather_scaled(const DevPool& p, const Batch& b, int32_t layer, int32_t H, int32_t D,
                                 const float* scales, int32_t type, void* out_k, void* out_v, cudaStream_t s);

// One attention call, as the kernels take it.
struct AttendArgs {
  const void* q;
  void* out;
  float* lse;           // or nullptr
  const float* scales;  // 8-bit pools, else nullptr
  int64_t q_stride;     // elements
  float scale_log2;     // softmax scale * log2(e)
  int32_t window;       // 0: none
  int32_t sinks;
  int32_t H, Q, D, G;   // G = Q / H
  int32_t layer;
  int32_t type;         // KV_TYPE_BF16 or KV_TYPE_F16, of q and out
};

// Set-up of the kernels on the current device (their shared-memory limits), of those
// that calls on a pool of this geometry can take (a pool more takes 84 us so, and 106 when
// all kernels are set up each time). Called by kv_pool_create.
cudaError_t prepare_append(const kv_pool_desc& d);
cudaError_t prepare_attend(const kv_pool_desc& d);
int64_t attend_workspace_bytes(int32_t H, int32_t Q, int32_t D, int32_t n_seqs, int64_t n_rows, int sm_count);
cudaError_t launch_attend(const DevPool& p, const Batch& b, const AttendArgs& a, bool e4m3, void* workspace,
                          int sm_count, cudaStream_t s);

// A launch that starts while the kernel before it drains (programmatic dependent launch).
template <class... A, class... B>
inline cudaError_t launch_overlapped(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                                     const B&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace gtkv
