// ops.h -- argument checks and per-device facts shared by the operators beside the codec: the 4-bit
// container (fp4.cu), its product (fp4_matmul.cu) and the quantised cache (cache.cu).
#pragma once

#include <cuda_runtime_api.h>

#include "entropack.h"

namespace ep {
namespace op {

constexpr int64_t kMaxFp4Cols = int64_t(1) << 30;
constexpr int64_t kMaxFp4Rows = (int64_t(1) << 31) - 256;

// The calling thread's current device and its SM count (looked up once per device).
int current_device(int& dev, int& sms);

// Format, sizes and pointers of a 4-bit tensor.
int check_fp4(const ep_fp4_tensor* t, const char* who);

}  // namespace op
}  // namespace ep
