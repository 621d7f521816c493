// Host helpers that the C-ABI files share (defined in api.cu).
#pragma once
#include <cuda.h>

#include <cstdint>

#include "../../include/kq.h"

namespace kq {

struct DeviceInfo { bool ok = false; int sms = 0; int device = 0; };

// The current device: KQ_ERR_NO_SM100 unless its compute capability is 10.0.
kq_status current_device(DeviceInfo* out);

// 2-D tiled tensor map: inner extent (elements), outer extent (rows), row pitch (bytes).
bool make_tmap(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner,
               uint64_t outer, uint64_t pitch, uint32_t box_inner, uint32_t box_outer,
               CUtensorMapSwizzle sw);

// 16-byte alignment of a caller's device pointer.
bool aligned(const void* p);

}  // namespace kq
