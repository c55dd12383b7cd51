// linear_mid.hip - y = x W^T on block codes, a matrix for all rows (linear_mid.h).
#include "linear_mid.h"

namespace zpp {

hipError_t launch_linear_mid(const LinArgs &p, int bits, bool a_f32, int mt, hipStream_t stream) {
    return launch_mid<LinMode::one>(p, bits, a_f32, mt, stream);
}

}  // namespace zpp
