// TMA tensor maps (defined in rkv_host.cpp).
#pragma once

#include <cstdint>
#include <cuda.h>

namespace rkv {

// 3D bf16 map, innermost dimension d = 128 elements, box {64, box1, box2}, 128-byte swizzle.
bool encode_map(CUtensorMap* m, const void* base, uint64_t dim1, uint64_t dim2, uint64_t stride1_bytes,
                uint64_t stride2_bytes, uint32_t box1, uint32_t box2);

}  // namespace rkv
