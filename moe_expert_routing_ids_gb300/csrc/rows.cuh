// What the kernels of quantised rows (8 bits, 4 bits) share.
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
// The 4-bit rows' border at k = 8 is the same or a little higher, to MX and NV, by position / by
// token: H = 4096, 4 MB 6.5 and 9.1 / 13 and 13 us, 8 MB 11 and 16 / 13 and 15, 16 MB 21 and 29 /
// 18 and 20; H = 1024, 4 MB 8.6 and 11 / 11 and 11, 8 MB 15 and 20 / 14 and 16; H = 128, 8 MB 18 and
// 23 / 19 and 21.  At k = 1 and 2 by position is the faster up to 16 MB at least (H = 4096, k = 2:
// 6.5 and 9.1 / 13 and 13): the rule does not ask for k.
constexpr int64_t kGatherBytes = 4 << 20;

// A sum of products times two float32 scales r and s, where r * s, or the sum times either, may be
// past float32's range though the result is not: first_factor(r), then s, then rest_factor(r),
// which is 1 unless r is beyond 2^-90 .. 2^77, and then about as far from 1 as the first, a
// power of two.  Sums of e2m1 values and e4m3 scales, or of f16 ones in their place, are 0 or
// within 2^-34 .. 2^45: neither step leaves float32's normal numbers where the result does not.
__device__ __forceinline__ int scale_exp(float r) { return (int)(__float_as_uint(r) >> 23 & 0xffu) - 127; }
__device__ __forceinline__ bool far_scale(float r) { return r != 0.f && (scale_exp(r) < -90 || scale_exp(r) >= 77); }
__device__ __forceinline__ float half_power(float r, int sign) { return __uint_as_float((uint32_t)(127 + sign * (scale_exp(r) / 2)) << 23); }
__device__ __forceinline__ float first_factor(float r) { return far_scale(r) ? half_power(r, 1) : r; }
__device__ __forceinline__ float rest_factor(float r) { return far_scale(r) ? r * half_power(r, -1) : 1.f; }
__device__ __forceinline__ float two_scales(float sum, float r, float s) { return sum * first_factor(r) * s * rest_factor(r); }

}  // namespace topo
