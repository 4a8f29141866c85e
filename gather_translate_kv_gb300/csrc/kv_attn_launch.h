// Host launchers of the operators of kv_attention.h; each enqueues on `s` and
// returns the launch status.
#pragma once

#include "kv_attention.h"
#include "kv_batch.cuh"

namespace gtkv {

// What the cache holds.
enum class Kind { kElements, kE4M3, kE2M1 };
inline Kind kind_of(const kv_pool_desc& d) {
  return d.format == KV_FORMAT_E2M1 ? Kind::kE2M1 : d.itemsize == 1 ? Kind::kE4M3 : Kind::kElements;
}

cudaError_t launch_append(const DevPool& p, const Batch& b, int32_t layer, int32_t type, Kind kind, int32_t H,
                          int32_t D, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const kv_rotary* rot, const void* q, int64_t q_stride, int32_t Q, void* q_out, float* scales,
                          int sm_count, cudaStream_t s);

cudaError_t launch_gather4(const DevPool& p, const Batch& b, int32_t layer, int32_t H, int32_t D, int32_t type,
                           void* out_k, void* out_v, cudaStream_t s);
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
  int32_t Gp;           // row f of a sequence is at its position a + f / Gp: G, or past all rows where they share one
  float* state = nullptr;        // not out and lse but what a row has summed up so far is written, [n_rows, Q] rows
  const float* prior = nullptr;  // what rows have summed up before; one of the two at most
  int64_t state_rows = 0;        // n_rows * Q: sums [state_rows][D], references [state_rows], denominators [state_rows]
};

// Set-up of the kernels on the current device (their shared-memory limits), of those
// that calls on a pool of this geometry can take. Called by kv_pool_create, but for the attention of shared prefixes, which a pool
// sets up at its first use.
cudaError_t prepare_append(const kv_pool_desc& d);
cudaError_t prepare_attend(const kv_pool_desc& d, bool shared);
int64_t attend_workspace_bytes(int32_t H, int32_t Q, int32_t D, int32_t n_seqs, int64_t n_rows, int sm_count);
// Attention of groups of sequences that share their first tokens.
int64_t attend_shared_workspace_bytes(int32_t Q, int32_t D, int32_t n_seqs, int64_t n_rows, int sm_count);
cudaError_t launch_attend_shared(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, const Groups& g,
                                 const int32_t* prefix_len, void* workspace, int sm_count, cudaStream_t s);
// Attention that shares nothing; groups, if there are any, are looked at.
cudaError_t launch_attend(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, const Groups& g,
                          void* workspace, int sm_count, cudaStream_t s);

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
