// The tiled products on 8-bit codes: y = x W^T.
#include "linear_tile.h"

namespace zpp {

hipError_t launch_linear_tile_fwd8(const LinArgs &p, int mode, int mt, hipStream_t stream) {
    return launch_linear_tile_as<false, 8>(p, mode, mt, stream);
}

}  // namespace zpp
