// dWg = dg^T x, dWu = du^T x of the gated feed-forward block (gated_ff_tile.hpp).
#include "gated_ff_tile.hpp"

namespace rar {

hipError_t launch_ff_dw(int dt, FfProduct& a, bool wide, bool direct, hipStream_t stream) {
  return ff_launch_kind<FF_DW>(dt, a, wide, direct, stream);
}

}  // namespace rar
