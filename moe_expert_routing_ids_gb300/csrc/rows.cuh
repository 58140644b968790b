// What the kernels that quantise rows (8 bits, 4 bits) share.
#pragma once

#include <cstdint>

namespace topo {

// 16 bf16 values.
__device__ __forceinline__ void unpack16(const uint4 &a, const uint4 &b, float (&v)[16]) {
    const uint32_t q[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(q[i] << 16);
        v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
}

// Up to this size the token rows of a dispatch are read k times, position by
// position (one launch), and not token by token through the inverse permutation
// (three).  k = 8, H = 4096, the call's launches included, by position / by token:
// 333 tokens 18.9 / 24.1 us, 1024 29.6 / 26.4, 4096 62.9 / 51.4, 16384 239 / 132.
// Both sides were measured at k = 8 only.  By token at k = 1, 2, 4 and 8, 16384 tokens:
// 52, 64, 83 and 124 us, against 30, 41, 61 and 103 for the bytes alone.
constexpr int64_t kGatherBytes = 4 << 20;

}  // namespace topo
