// k_attend_tile for 16-bit caches.
#include "kv_attend_tile.cuh"

namespace gtkv {

GTKV_TILE_INSTANCES(__half, false)
GTKV_TILE_INSTANCES(__nv_bfloat16, false)

}  // namespace gtkv
