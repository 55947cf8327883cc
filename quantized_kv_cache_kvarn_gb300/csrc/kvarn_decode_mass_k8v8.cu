// Decode kernels that gather tile masses: K8V8, fp16 scales.
#include "kvarn_decode_kernel.cuh"

namespace kvarn {
KVARN_DECODE_MASS(8, 8, 2)
}  // namespace kvarn
