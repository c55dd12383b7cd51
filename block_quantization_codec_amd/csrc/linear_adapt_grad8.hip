// The tiled products on 8-bit codes, rows with low-rank adapters (linear_adapt.h): dx = dy W.
// 4096 rows of 8192 x 8192 with one adapter of rank 64: 475 us, against 461 without adapters.
#include "linear_big.h"

namespace zpp {

hipError_t launch_linear_adapt_grad8(const LinArgs &p, int parts, int mt, hipStream_t stream) {
    return launch_linear_big_as<LinMode::adapted, true, 8>(p, parts, mt, stream);
}

}  // namespace zpp
