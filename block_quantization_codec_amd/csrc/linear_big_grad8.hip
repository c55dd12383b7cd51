// The tiled products on 8-bit codes: dx = dy W.
#include "linear_big.h"

namespace zpp {

hipError_t launch_linear_big_grad8(const LinArgs &p, int parts, int mt, hipStream_t stream) {
    return launch_linear_big_as<true, 8>(p, parts, mt, stream);
}

}  // namespace zpp
