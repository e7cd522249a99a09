// Host-side checks shared by the translation units that hold entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "../../include/ps.h"

namespace ps {

constexpr size_t kAlign = 256;              // workspace alignment

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Bytes of an element of a ps_dtype; 0 for any other value.
int elem_size(int32_t dtype);
// Whether `ptr` is memory that kernels may be given: a device's, or managed.
bool on_device(const void *ptr);
// Makes the device that owns `ptr` current; its SM count.
ps_status device_of(const void *ptr, int *sms);
ps_status map_cuda(cudaError_t e);
bool aligned(const void *p, size_t a);
int32_t integer_power(double tau);
ps_status check_batch_host(const ps_subtree_batch *b, bool need_data = true);

}  // namespace ps
