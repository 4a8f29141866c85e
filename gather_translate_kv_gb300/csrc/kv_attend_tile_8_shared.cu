// k_attend_tile for 8-bit caches, shared prefixes.
#include "kv_attend_tile.cuh"

namespace gtkv {

GTKV_TILE_INSTANCES(CodeE4M3, true)

}  // namespace gtkv
