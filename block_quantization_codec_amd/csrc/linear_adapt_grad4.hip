// The tiled products on 4-bit codes, rows with low-rank adapters (linear_adapt.h): dx = dy W.
#include "linear_big.h"

namespace zpp {

hipError_t launch_linear_adapt_grad4(const LinArgs &p, int parts, int mt, hipStream_t stream) {
    return launch_linear_big_as<LinMode::adapted, true, 4>(p, parts, mt, stream);
}

}  // namespace zpp
