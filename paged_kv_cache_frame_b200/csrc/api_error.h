// What the files of C entry points share: the calling thread's last error,
// and the current device's SM count.
#pragma once
#include <cuda_runtime.h>

#include <string>

namespace pkv {

// Records `why` for kv_last_error and returns `code`.
int api_fail(int code, const std::string& why);
// KV_ERR_CUDA, with CUDA's text.
int api_cuda_fail(cudaError_t e, const char* where);
int current_device_sms();

}  // namespace pkv
