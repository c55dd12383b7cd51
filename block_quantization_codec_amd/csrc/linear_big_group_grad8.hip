// The tiled products on 8-bit codes, a matrix for each group of rows: dx = dy W.
// 4096 rows over 8 matrices of 11008 x 4096 with unequal shares: 394 to 414 us, 14 of them the join.
// Matrix instructions and the codes' conversion bound it; last tiles are not full.
#include "linear_big.h"

namespace zpp {

hipError_t launch_linear_big_group_grad8(const LinArgs &p, int parts, int mt, hipStream_t stream) {
    return launch_linear_big_as<LinMode::grouped, true, 8>(p, parts, mt, stream);
}

}  // namespace zpp
