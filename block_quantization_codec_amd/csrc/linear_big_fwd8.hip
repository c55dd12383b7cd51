// The tiled products on 8-bit codes: y = x W^T.
#include "linear_big.h"

namespace zpp {

hipError_t launch_linear_big_fwd8(const LinArgs &p, int parts, int mt, hipStream_t stream) {
    return launch_linear_big_as<false, 8>(p, parts, mt, stream);
}

}  // namespace zpp
