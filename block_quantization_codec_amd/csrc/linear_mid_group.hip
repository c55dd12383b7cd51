// linear_mid_group.hip - y = x W^T on block codes, a matrix for each group of rows (linear_mid.h).
// Memory bounds it: 32 rows over 16 matrices of 11008 x 4096 int4, 79 to 87 us with the join
// (the codes of the matrices that have rows: 59 us as a copy).
#include "linear_mid.h"

namespace zpp {

hipError_t launch_linear_mid_group(const LinArgs &p, int bits, bool a_f32, int mt, hipStream_t stream) {
    return launch_mid<LinMode::grouped>(p, bits, a_f32, mt, stream);
}

}  // namespace zpp
