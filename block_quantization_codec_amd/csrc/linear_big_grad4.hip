// The tiled products on 4-bit codes: dx = dy W.
#include "linear_big.h"

namespace zpp {

hipError_t launch_linear_big_grad4(const LinArgs &p, int parts, int mt, hipStream_t stream) {
    return launch_linear_big_as<true, 4>(p, parts, mt, stream);
}

}  // namespace zpp
