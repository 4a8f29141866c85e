// k_attend_few for 16-bit caches, shared prefixes.
#include "kv_attend_few.cuh"

namespace gtkv {

GTKV_FEW_INSTANCES(__half, true)
GTKV_FEW_INSTANCES(__nv_bfloat16, true)

}  // namespace gtkv
