// Decode kernels that gather tile masses: K6V6, fp16 scales.
#include "kvarn_decode_kernel.cuh"

namespace kvarn {
KVARN_DECODE_MASS(6, 6, 2)
}  // namespace kvarn
