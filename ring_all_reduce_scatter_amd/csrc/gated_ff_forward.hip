// h = act(x Wg^T) (x Wu^T) of the gated feed-forward block (gated_ff_tile.hpp).
#include "gated_ff_tile.hpp"

namespace rar {

hipError_t launch_ff_forward_tiles(int dt, FfProduct& a, bool wide, bool direct, hipStream_t stream) {
  return ff_launch_kind<FF_FORWARD>(dt, a, wide, direct, stream);
}

}  // namespace rar
