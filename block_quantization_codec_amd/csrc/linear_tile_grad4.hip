// The tiled products on 4-bit codes: dx = dy W.
#include "linear_tile.h"

namespace zpp {

hipError_t launch_linear_tile_grad4(const LinArgs &p, int mode, int mt, hipStream_t stream) {
    return launch_linear_tile_as<true, 4>(p, mode, mt, stream);
}

}  // namespace zpp
