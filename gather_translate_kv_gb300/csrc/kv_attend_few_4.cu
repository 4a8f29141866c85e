// k_attend_few for 4-bit caches.
#include "kv_attend_few.cuh"

namespace gtkv {

GTKV_FEW_INSTANCES(CodeE2M1, false)

}  // namespace gtkv
