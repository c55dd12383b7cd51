// The tiled products on 4-bit codes: y = x W^T.
#include "linear_tile.h"

namespace zpp {

hipError_t launch_linear_tile_fwd4(const LinArgs &p, int mode, int mt, hipStream_t stream) {
    return launch_linear_tile_as<false, 4>(p, mode, mt, stream);
}

}  // namespace zpp
