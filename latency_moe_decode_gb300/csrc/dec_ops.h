// Host helpers shared by the operator entry points (dec_kvq.cu, dec_logprobs.cu) and the engine.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "dec.h"

namespace dec {

// The calling thread's operator error text (dec_op_error).
dec_status op_fail(dec_status s, const char* msg);
dec_status op_cuda(cudaError_t c, const char* what);
void op_clear();

// Streaming multiprocessors of the current device (looked up once per device).
int op_sms();
// DEC_ERR_ARG unless p is device memory of the current device.
dec_status op_on_device(const void* p, const char* what);

inline cudaStream_t op_stream(void* s) { return s ? static_cast<cudaStream_t>(s) : cudaStreamLegacy; }
inline bool op_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace dec
