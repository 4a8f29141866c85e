// k_attend_tile for 4-bit caches, shared prefixes.
#include "kv_attend_tile.cuh"

namespace gtkv {

GTKV_TILE_INSTANCES(CodeE2M1, true)

}  // namespace gtkv
