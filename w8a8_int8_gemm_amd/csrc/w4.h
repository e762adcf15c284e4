// w4.h -- launchers of the 4-bit linear and its converters (w4.hip).  Not part
// of the public ABI (include/w8a8.h); arguments are validated by the API layer
// before.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {

hipError_t launch_w4_quantize(const uint16_t *w, int64_t N, int64_t K,
                              int group, uint8_t *w4, uint16_t *scale,
                              hipStream_t stream);
hipError_t launch_w4_pack(const int8_t *codes, const uint16_t *scales,
                          int64_t N, int64_t K, int group, uint8_t *w4,
                          uint16_t *scale, hipStream_t stream);
hipError_t launch_w4_linear(const uint16_t *x, const uint8_t *w4,
                            const uint16_t *scale, const uint16_t *bias,
                            uint16_t *y, int64_t M, int64_t N, int64_t K,
                            int group, hipStream_t stream);

}  // namespace w8a8
