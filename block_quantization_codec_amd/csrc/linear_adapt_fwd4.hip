// The tiled products on 4-bit codes, rows with low-rank adapters (linear_adapt.h): y = x W^T.
// 4096 rows of 8192 x 28672 with 4 adapters of rank 64: 1608 us, against 1536 without adapters.
#include "linear_big.h"

namespace zpp {

hipError_t launch_linear_adapt_fwd4(const LinArgs &p, int parts, int mt, hipStream_t stream) {
    return launch_linear_big_as<LinMode::adapted, false, 4>(p, parts, mt, stream);
}

}  // namespace zpp
