// The kernel of few rows a sequence (kv_attend_few.cuh) for 4-bit caches.
#include "kv_attend_few.cuh"

namespace gtkv {

cudaError_t prepare_few4(int32_t D, bool p16) { return prepare_c<CodeE2M1>(D, p16); }

cudaError_t launch_few4(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w, int nt, bool after,
                        cudaStream_t s) {
  return launch_c<CodeE2M1>(p, b, a, w, nt, after, s);
}

}  // namespace gtkv
