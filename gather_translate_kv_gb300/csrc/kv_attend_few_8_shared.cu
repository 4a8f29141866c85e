// k_attend_few for 8-bit caches, shared prefixes.
#include "kv_attend_few.cuh"

namespace gtkv {

GTKV_FEW_INSTANCES(CodeE4M3, true)

}  // namespace gtkv
