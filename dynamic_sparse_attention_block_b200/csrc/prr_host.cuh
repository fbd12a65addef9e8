// prr_host.cuh -- host-side helpers shared by the translation units that implement the
// C ABI: shape rules, kernel parameters, tensor maps, device properties.
#pragma once

#include "prr.h"
#include "prr_kernels.cuh"

namespace prr {

struct DeviceInfo {
  int sms = 0;
  int prio_high = 0, prio_low = 0;
};

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline prr_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PRR_OK : PRR_ERR_CUDA; }

bool dims_ok(const prr_dims* d);
DeviceInfo device_info();
Params base_params(const prr_dims* d, void* ws, bool kv_units = false);
bool make_kv_map(CUtensorMap* map, const void* base, const prr_dims* d);
bool make_kv_step_map(CUtensorMap* map, const void* base, const prr_dims* d);
bool make_q_map(CUtensorMap* map, const void* base, int64_t stride, int32_t rows, const prr_dims* d);

}  // namespace prr
