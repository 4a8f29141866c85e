// k_attend_tile for 4-bit caches.
#include "kv_attend_tile.cuh"

namespace gtkv {

GTKV_TILE_INSTANCES(CodeE2M1, false)

}  // namespace gtkv
