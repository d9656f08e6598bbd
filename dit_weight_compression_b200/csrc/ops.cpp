// ops.cpp -- see ops.h.
#include "ops.h"

#include <atomic>
#include <string>

#include "blob.h"

namespace ep {
namespace op {

int current_device(int& dev, int& sms) {
    static std::atomic<int> count[kMaxDevices];
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevices)) return set_error(EP_ERR_ARG, "device ordinal out of range");
    if (e == cudaSuccess) {
        sms = count[dev].load(std::memory_order_relaxed);
        if (sms == 0) {
            e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            if (e == cudaSuccess) count[dev].store(sms, std::memory_order_relaxed);
        }
    }
    if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("current device: ") + cudaGetErrorString(e));
    return EP_OK;
}

int check_fp4(const ep_fp4_tensor* t, const char* who) {
    const std::string w(who);
    if (t->format != EP_MXFP4 && t->format != EP_NVFP4) return set_error(EP_ERR_DTYPE, w + ": not a 4-bit format");
    if (t->rows < 0 || t->cols < 0 || t->rows > kMaxFp4Rows || t->cols > kMaxFp4Cols)
        return set_error(EP_ERR_SHAPE, w + ": 4-bit tensor size out of range");
    if (!t->tensor_scale || reinterpret_cast<uintptr_t>(t->tensor_scale) % 4)
        return set_error(EP_ERR_ARG, w + ": the 4-bit tensor's tensor_scale is NULL or misaligned");
    if (t->rows > 0 && t->cols > 0) {
        if (!t->data || !t->scales) return set_error(EP_ERR_ARG, w + ": the 4-bit tensor has no data or scales");
        if (reinterpret_cast<uintptr_t>(t->data) % 16 || reinterpret_cast<uintptr_t>(t->scales) % 16)
            return set_error(EP_ERR_ARG, w + ": 4-bit data and scales must be 16-byte aligned");
    }
    return EP_OK;
}

}  // namespace op
}  // namespace ep
