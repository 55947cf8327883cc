// Decode kernels that gather tile masses: K4V4, fp16 scales.
#include "kvarn_decode_kernel.cuh"

namespace kvarn {
KVARN_DECODE_MASS(4, 4, 2)
}  // namespace kvarn
