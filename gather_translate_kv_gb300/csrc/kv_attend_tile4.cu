// The kernel of many rows a sequence (kv_attend_tile.cuh) for 4-bit caches.
#include "kv_attend_tile.cuh"

namespace gtkv {

cudaError_t prepare_tile4(int32_t D) {
  const cudaError_t e = prepare_one<CodeE2M1, false, false>(D);
  return e == cudaSuccess ? prepare_one<CodeE2M1, false, true>(D) : e;
}

cudaError_t launch_tile4(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w, bool after, cudaStream_t s) {
  return a.type == KV_TYPE_BF16 ? launch_one<CodeE2M1, false, false>(p, b, a, w, after, s)
                                : launch_one<CodeE2M1, false, true>(p, b, a, w, after, s);
}

}  // namespace gtkv
