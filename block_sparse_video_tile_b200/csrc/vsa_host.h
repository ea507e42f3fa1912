// vsa_host.h -- host helpers that libvsa.so's translation units share.
#pragma once

#include <cstdint>

namespace vsa {

// VSA_OK if the current device is sm_100 (defined in libvsa.cu).
int check_arch();
// Device address of the kernels' error word on the current device, or nullptr
// (defined in libvsa.cu).
unsigned int* device_error_ptr();

inline bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }

// Strides (b, n, h) of a strided tensor with extents B, N, H and d channels:
// positive multiples of 8 elements; those of an extent of 1 are never used
// and become d.  Returns a vsa_status.
int take_strides(const int64_t in[3], int B, int N, int H, int d, long long out[3]);

}  // namespace vsa
