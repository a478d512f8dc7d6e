// Host-side helpers of the C-ABI layer that entry points in other translation units share.
#pragma once
#include <cuda.h>
#include <cstdint>

namespace fa {

// 4-D bf16 tensor map with 128-byte swizzle; dims innermost first, strides in bytes for dims 1..3.
bool make_bf16_map(CUtensorMap* m, const void* base, const uint64_t dims[4], const uint64_t strides[3],
                   const uint32_t box[4]);

inline bool is_aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Whether two memory ranges share a byte.
inline bool overlaps(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + b_bytes && y < x + a_bytes;
}

}  // namespace fa
