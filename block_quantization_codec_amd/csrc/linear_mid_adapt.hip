// linear_mid_adapt.hip - y = x W^T on block codes, and each row's adapter beside it (linear_mid.h).
#include "linear_mid.h"

namespace zpp {

hipError_t launch_linear_mid_adapt(const LinArgs &p, int bits, bool a_f32, int mt, hipStream_t stream) {
    return launch_mid<LinMode::adapted>(p, bits, a_f32, mt, stream);
}

}  // namespace zpp
