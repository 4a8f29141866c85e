// k_attend_tile for 16-bit caches, shared prefixes.
#include "kv_attend_tile.cuh"

namespace gtkv {

GTKV_TILE_INSTANCES(__half, true)
GTKV_TILE_INSTANCES(__nv_bfloat16, true)

}  // namespace gtkv
