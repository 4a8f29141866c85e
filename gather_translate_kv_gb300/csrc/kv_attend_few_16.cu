// k_attend_few for 16-bit caches.
#include "kv_attend_few.cuh"

namespace gtkv {

GTKV_FEW_INSTANCES(__half, false)
GTKV_FEW_INSTANCES(__nv_bfloat16, false)

}  // namespace gtkv
