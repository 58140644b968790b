// Rows in microscaled 4 bits: e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), two to a byte, with a scale for each block of a row.
//
//   MX  blocks of 32, the scale a power of two as its exponent (UE8M0):
//       s = the smallest 2^n with amax <= 6 s
//   NV  blocks of 16, the scale in e4m3, over a power of two g for the whole row:
//       g = the smallest 2^n with row amax <= 6 * 448 g,
//       s = the smallest e4m3 value with amax <= 6 s g
//
// (n >= -126; 1 for zeros) and q = e2m1(v / s) or e2m1(v / (s g)), to nearest, ties
// to even: no value is clipped.  A block that holds a NaN or an infinity gets the
// scale NaN.  Division by a power of two is exact.  With an e4m3 scale of 4 bits, a bf16
// value's quotient is a border between two values of e2m1 (at most 3 bits) or at least
// 2^-8 of it away: the product with the scale's inverse, within 2^-22, rounded to f16 is
// on the right side, or on the border.  The activation's quotients, of float32 values, are
// left as they are, within 2^-22.
//
//   k_micro_rows     rows as they are, dispatch rows (by position, or token row t to the
//                    k layout positions of its pairs), or the gated activation
//                    silu(g) * u of rows [g | u]
//   k_micro_narrow   the same for rows of up to 512 values, several to a warp
//   k_micro_values   the bf16 values that such rows stand for
//
// A lane takes 16 consecutive values (32 bytes in, 8 bytes out): a block of NV, half
// a block of MX.  Measured, bytes moved over time: rows of 131072 x 7168 to MX 332 us,
// 7.2 TB/s, to NV 397 us, 6.1 TB/s (the row's largest value first, its words in registers
// meanwhile: issue 70 percent); weights of 64 x 2816 x 4096 to MX 256 us, 7.3 TB/s, and back
// to bf16 266 us; activation of 131072 x 2048 to MX 192 us, 6.3 TB/s, to NV 235 us, 5.2 TB/s
// (issue 74 percent); dispatch of 16384 tokens, k = 8, H = 7168 to NV 145 us and 5 us for the
// inverse permutation.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "rows.cuh"

namespace topo {
namespace {

enum { kPlain = 0, kScatter = 1, kSwiglu = 2, kGather = 3 };

constexpr uint32_t kInf = 0x7f800000u;

__device__ __forceinline__ float pow2(int n) { return __uint_as_float((uint32_t)(127 + n) << 23); }   // -126 .. 127

// Exponent of the smallest power of two s with amax <= m * 2^p * s, m in [1, 2) given
// by its fraction bits; amax by its bits, finite.
__device__ __forceinline__ int least_power(uint32_t amax, uint32_t frac, int p) {
    const int n = (int)(amax >> 23) - 127 - p + ((amax & 0x7fffffu) > frac ? 1 : 0);
    return amax == 0u ? 0 : max(n, -126);
}

// The value of an e4m3 byte (one that is no NaN).
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
    return __half2float(__ushort_as_half((unsigned short)h));
}

// Eight values in 4 bits, the first in the lowest.  HALF: through f16, whose 11 bits hold
// every border between two values of e2m1.
template <bool HALF>
__device__ __forceinline__ uint32_t e2m1x8(const float *v) {
    uint32_t r;
    if (HALF) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            h[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f16x2 a, %1;\n cvt.rn.satfinite.e2m1x2.f16x2 b, %2;\n"
            " cvt.rn.satfinite.e2m1x2.f16x2 c, %3;\n cvt.rn.satfinite.e2m1x2.f16x2 d, %4;\n mov.b32 %0, {a, b, c, d};\n}\n"
            : "=r"(r)
            : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
    } else {
        asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
            " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
            : "=r"(r)
            : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    }
    return r;
}

struct MicroArgs {
    const uint4 *x;          // bf16 rows, two uint4 per 16 values
    const int32_t *inv;      // kScatter: position of each pair; kGather: pair of each position
    uint2 *q;                // packed rows, 8 bytes per 16 values
    uint8_t *scale;          // [rows][pitch]
    float *row_scale;        // NV: [rows]
    WsHeader *hdr;
    int64_t rows;            // rows over all layers (kGather: output rows)
    int64_t npairs;
    int T, k;                // kScatter, kGather: tokens per layer, copies of a row
    int nv;                  // 16-value groups per (output) row
    int pitch;
    int log_w;               // a row is split over 2^log_w warps, at most 8
    int log_l;               // k_micro_narrow: a row takes 2^log_l lanes
};

// Bits of the largest finite magnitude of 16 values.
__device__ __forceinline__ uint32_t finite_bits(const float (&v)[16]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
        if (u < kInf) m = max(m, u);
    }
    return m;
}

// Two float32 values in a register pair, for the packed instructions.
using f2 = uint64_t;
__device__ __forceinline__ f2 pair(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 both(float a) { return pair(a, a); }
__device__ __forceinline__ void halves(f2 p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// v = silu(v) * u in float32.  exp(-v) as a power of two of the rounded product t =
// -v log2(e), times 1 + what the rounding left out; the reciprocal of 1 + exp(-v) by one
// step of Newton's iteration from the approximate one: within 8 * 2^-24 of the value, where
// topo_swiglu_quantize calls expf and divides (25 instructions a value; this, in packed
// pairs, 9).  far: some |v| may be above 83: expf and division.  (Below -83 1 + exp(-v)
// nears the end of float32's range, above 2.35e38 v log2(e) is past it.  A bound of its own for
// either sign costs a second maximum: 131072 x 2048 to MX and NV 189 and 234 us with the one for
// -83 alone, 194 and 240 with both, 191 and 235 with this one.)
__device__ __forceinline__ void gated(float (&v)[16], const float (&u)[16], bool far) {
    if (far) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __fdiv_rn(v[i], 1.f + expf(-v[i])) * u[i];
        return;
    }
    constexpr double kLog2e = 1.44269504088896341;               // in two parts
    const f2 to = both(-(float)kLog2e), back = both((float)kLog2e), lo = both((float)((float)kLog2e - kLog2e));
    const f2 ln2 = both(0.69314718f), one = both(1.f), less = both(-1.f);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const f2 x = pair(v[i], v[i + 1]), t = mul2(x, to), left = fma2(lo, x, fma2(to, x, mul2(x, back)));   // x back = -t
        float t0, t1, e0, e1, r0, r1;
        halves(t, t0, t1);
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t0));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t1));
        const f2 e = pair(e0, e1), c = fma2(mul2(e, ln2), left, e), nd = fma2(c, less, less);   // -(1 + exp(-v))
        halves(nd, r0, r1);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(-r0));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(-r1));
        const f2 r = pair(r0, r1);
        halves(mul2(mul2(x, fma2(fma2(nd, r, one), r, r)), pair(u[i], u[i + 1])), v[i], v[i + 1]);
    }
}

// A lane's groups of a row: kGroups of them, 32 apart, at a time, kept as they are stored
// (the activation's as float32).
// Measured in groups, CTAs to an SM: activation of 131072 x 2048 to MX 1, 4: 221 us, 1, 5: 231,
// 2, 3: 204, 2, 4: 193, 3, 2: 310; to NV 1, 5: 296, 2, 3: 246, 2, 4: 236; rows of 131072 x 7168 to
// NV 4, 3: 429, 4, 4: 399, 5, 3: 458.  run_rows takes the activation's three, 3 CTAs, where
// they need half as many warps.  At four CTAs' 64 registers rows to NV keep 13 or 14 words in
// local memory, narrow ones by token 13 (to MX 2), the activation to NV 4, of three groups 8.
template <int SRC>
constexpr int kGroups = SRC == kSwiglu ? 2 : 4;
constexpr int ctas(int src, int n) { return src == kSwiglu && n == 3 ? 3 : 4; }   // to an SM

template <int SRC, int N>
struct Groups {
    static constexpr int kN = N;
    uint4 a[kN][2];

    // Group j at src(j), zeros where in(j) is false.
    template <class Src, class In, class Any>
    __device__ __forceinline__ void load(int, Src src, In in, Any) {
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) a[j][i] = in(j) ? __ldg(src(j) + i) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(int j, float (&v)[16]) const { unpack16(a[j][0], a[j][1], v); }
    // Bits (float32) of the largest magnitude of group j, as NaN > infinity > finite values.
    __device__ __forceinline__ uint32_t amax(int j) const {
        const uint32_t w[8] = {a[j][0].x, a[j][0].y, a[j][0].z, a[j][0].w, a[j][1].x, a[j][1].y, a[j][1].z, a[j][1].w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        return max(m << 16, m & 0xffff0000u);
    }
};
template <int N>
struct Groups<kSwiglu, N> {
    static constexpr int kN = N;
    float f[kN][16];

    // any(j), the same for the whole warp: a lane has a group j.
    template <class Src, class In, class Any>
    __device__ __forceinline__ void load(int nv, Src src, In in, Any any) {
        uint4 a[kN][4];
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) a[j][i] = in(j) ? __ldg(src(j) + (i < 2 ? 0 : 2 * nv) + (i & 1)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            if (!any(j)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) f[j][i] = 0.f;
                continue;
            }
            const uint32_t w[8] = {a[j][0].x, a[j][0].y, a[j][0].z, a[j][0].w, a[j][1].x, a[j][1].y, a[j][1].z, a[j][1].w};
            const __nv_bfloat162 *const p = reinterpret_cast<const __nv_bfloat162 *>(w);
            __nv_bfloat162 most = __habs2(p[0]);                // the largest magnitudes; drops a NaN
#pragma unroll
            for (int i = 1; i < 8; ++i) most = __hmax2(most, __habs2(p[i]));
            const uint32_t bits = *reinterpret_cast<const uint32_t *>(&most);
            float u[16];
            unpack16(a[j][0], a[j][1], f[j]);
            unpack16(a[j][2], a[j][3], u);
            gated(f[j], u, max(bits & 0xffffu, bits >> 16) > 0x42a6u);   // 83
        }
    }
    __device__ __forceinline__ void get(int j, float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = f[j][i];
    }
    __device__ __forceinline__ uint32_t amax(int j) const {
        float m = 0.f;                                          // drops a NaN: 0 * v tells of those
        f2 z = both(0.f);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            m = fmaxf(fmaxf(m, fabsf(f[j][i])), fabsf(f[j][i + 1]));
            z = fma2(pair(f[j][i], f[j][i + 1]), both(0.f), z);
        }
        float a, b;
        halves(z, a, b);
        return a + b == 0.f ? __float_as_uint(m) : 0x7fffffffu;
    }
};

// A block's scale byte, v divided by the scale.  m: bits of the 16 values' largest magnitude,
// n: NV: exponent of the row's scale.
template <bool NV>
__device__ __forceinline__ uint32_t to_block(float (&v)[16], uint32_t m, int n) {
    uint32_t sb;
    if (NV) {
        // t / 6, at most 448, rounded up to e4m3 (the quotient's last bits are cut, so that
        // 6 times a scale gives the scale): a mantissa of 3 bits, or a multiple of 2^-9
        const float t = __fmul_rz(__uint_as_float(m) * pow2(-n), 1.f / 6.f);
        const uint32_t up = __float_as_uint(t) + 0xfffffu, low = __float_as_uint(__fadd_ru(t, 0x1p14f));
        float s = __uint_as_float(up & 0xfff00000u);
        sb = (up >> 20) - 960;
        if (t < 0x1p-6f) {
            s = fmaxf(__uint_as_float(low) - 0x1p14f, 0x1p-9f);   // t may underflow
            sb = max(low & 0xffu, 1u);
        }
        if (m == 0u) s = 1.f, sb = 0x38u;
        if (n < -112) {                                  // 1 / (s g) might be past float32's range
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= 0x1p16f;
        }
        const float sg = s * pow2(n < -112 ? n + 16 : n);
        float si;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(si) : "f"(sg));
#pragma unroll
        for (int i = 0; i < 16; i += 2) halves(mul2(pair(v[i], v[i + 1]), both(si)), v[i], v[i + 1]);
        if (m >= kInf) sb = 0x7fu;
    } else {
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        n = m < kInf ? least_power(m, 0x400000u, 2) : 0;   // 6 = 1.5 * 2^2
        const float inv = pow2(-n);
#pragma unroll
        for (int i = 0; i < 16; i += 2) halves(mul2(pair(v[i], v[i + 1]), both(inv)), v[i], v[i + 1]);
        sb = m < kInf ? (uint32_t)(127 + n) : 255u;
    }
    return sb;
}

// 2^log_w warps take a row, each kGroups * 32 groups of 16 values side by side; a row that
// is longer than eight warps' goes round (NV: and is read twice, once for its largest
// magnitude).  All of a lane's loads are on their way before the first is used.
template <int SRC, bool NV, int N>
__global__ void __launch_bounds__(256, ctas(SRC, N))
k_micro_rows(MicroArgs g) {
    constexpr int kPer = N * 32;
    __shared__ uint32_t wmax[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp & ((1 << g.log_w) - 1);
    const int64_t row = ((int64_t)blockIdx.x * 8 + warp) >> g.log_w;
    bool live = row < g.rows;                                    // the same for a row's warps
    int pa = 0, pb = 0;
    int64_t base = 0, from = row;
    pdl_trigger();
    pdl_wait();
    if (SRC == kGather && live) {
        const int64_t l = row / g.npairs;
        const int p = __ldg(g.inv + row);
        if ((uint64_t)p >= (uint64_t)g.npairs) {
            if (lane == 0) set_error(g.hdr, TOPO_ESTATE);
            live = false;
        }
        from = l * g.T + p / g.k;
    }
    if (SRC == kScatter && live) {
        base = (row / g.T) * g.npairs;
        const int32_t *iv = g.inv + row * g.k;
        pa = lane < g.k ? __ldg(iv + lane) : 0;
        pb = lane + 32 < g.k ? __ldg(iv + lane + 32) : 0;
        if (!__all_sync(0xffffffffu, (uint64_t)pa < (uint64_t)g.npairs && (uint64_t)pb < (uint64_t)g.npairs)) {
            if (lane == 0) set_error(g.hdr, TOPO_ESTATE);
            live = false;
        }
    }
    if (!live) from = 0;
    const int first = part * kPer + lane, span = kPer << g.log_w;
    const int nv = live ? (g.nv + 31) & ~31 : 0;                 // whole warps of groups
    Groups<SRC, N> in_regs;
    const uint4 *const src = g.x + from * ((SRC == kSwiglu ? 4 : 2) * (int64_t)g.nv);
    const auto load = [&](int c0) {
        in_regs.load(g.nv, [&](int j) { return src + 2 * (c0 + 32 * j); }, [&](int j) { return c0 + 32 * j < g.nv; },
                     [](int) { return true; });
    };
    float v[16];
    uint32_t am[N];                                   // the groups' largest magnitudes
    int n = 0;                                                   // NV: exponent of the row's scale
    if (NV) {
        // the whole row's largest finite magnitude first
        uint32_t m = 0;
        for (int c0 = first; c0 - lane < nv; c0 += span) {
            load(c0);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                am[j] = in_regs.amax(j);
                uint32_t a = am[j];
                if (a >= kInf) {
                    in_regs.get(j, v);
                    a = finite_bits(v);
                }
                m = max(m, a);
            }
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (g.log_w > 0) {
            if (lane == 0) wmax[warp] = m;
            __syncthreads();
            m = 0;
            for (int i = 0; i < 1 << g.log_w; ++i) m = max(m, wmax[(warp & ~((1 << g.log_w) - 1)) + i]);
        }
        n = least_power(m, 0x280000u, 11);                       // 6 * 448 = 1.3125 * 2^11
        if (SRC == kScatter && live && part == 0) {
            if (lane < g.k) g.row_scale[base + pa] = pow2(n);
            if (lane + 32 < g.k) g.row_scale[base + pb] = pow2(n);
        } else if (live && lane == 0 && part == 0) {
            g.row_scale[row] = pow2(n);
        }
    }
    for (int c0 = first; c0 - lane < nv; c0 += span) {
        if (!NV || g.nv > span) {
            load(c0);
#pragma unroll
            for (int j = 0; j < N; ++j) am[j] = in_regs.amax(j);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = c0 + 32 * j;
            if (c - lane >= nv) break;                           // whole warp
            const bool in = c < g.nv;
            in_regs.get(j, v);
            uint32_t sb = to_block<NV>(v, am[j], n);
            constexpr bool kHalf = NV && SRC != kSwiglu;
            const uint2 q = make_uint2(e2m1x8<kHalf>(v), e2m1x8<kHalf>(v + 8));
            // four blocks' scales to a word, on the first of their lanes; bytes past the last
            // block hold 1
            constexpr int kLanes = NV ? 4 : 8;                   // lanes of a word
            sb |= __shfl_down_sync(0xffffffffu, sb, kLanes / 4) << 8;
            sb |= __shfl_down_sync(0xffffffffu, sb, kLanes / 2) << 16;
            const int at = c / kLanes * 4;
            const bool word = lane % kLanes == 0 && at < g.pitch;
            if (SRC == kScatter) {
                for (int i = 0; i < g.k; ++i) {
                    const int a = __shfl_sync(0xffffffffu, pa, i & 31), b = __shfl_sync(0xffffffffu, pb, i & 31);
                    const int64_t r = base + (i < 32 ? a : b);
                    if (in) g.q[r * g.nv + c] = q;
                    if (word) *reinterpret_cast<uint32_t *>(g.scale + r * g.pitch + at) = sb;
                }
            } else {
                if (in) g.q[row * g.nv + c] = q;
                if (word) *reinterpret_cast<uint32_t *>(g.scale + row * g.pitch + at) = sb;
            }
        }
    }
}

// Rows of at most 32 groups: 2^log_l lanes take one, the groups of a lane are of kGroups
// rows, 32 / 2^log_l apart, so that all lanes have work and as many loads on their way as
// with a longer row.  131072 rows to MX / NV, against a warp for each row: of 128 values 6.7 /
// 9.2 us and 36.7 / 53.1 (6.6 / 4.8 TB/s), of 512 values 27.4 / 34.6 and 42.4 / 57.8; activation
// of 512 values 54 / 61 and 85 / 100; dispatch of 16384 tokens by token, k = 8, of 128 values
// 10.0 / 12.7 and 47.1 / 66.5.
template <int SRC, bool NV>
__global__ void __launch_bounds__(256, 4)
k_micro_narrow(MicroArgs g) {
    constexpr int kN = kGroups<SRC>;
    constexpr int kLanes = NV ? 4 : 8;                           // lanes of a word of scales
    constexpr uint32_t kOne = NV ? 0x38u : 127u;                 // the scale 1
    const int lane = threadIdx.x & 31, lanes = 1 << g.log_l, sub = lane & (lanes - 1), apart = 32 >> g.log_l;
    const int64_t row0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * (kN * apart) + (lane >> g.log_l);
    const uint32_t mine = (0xffffffffu >> (32 - lanes)) << (lane - sub);   // the row's lanes
    const uint4 *src[kN];
    const int32_t *inv[kN];                                      // kScatter: the token's positions
    int64_t base[kN];
    bool live[kN];
    pdl_trigger();
    pdl_wait();
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        const int64_t row = row0 + j * apart;
        int64_t from = row;
        live[j] = row < g.rows;
        if (SRC == kGather && live[j]) {
            const int p = __ldg(g.inv + row);
            if ((uint64_t)p >= (uint64_t)g.npairs) {
                if (sub == 0) set_error(g.hdr, TOPO_ESTATE);
                live[j] = false;
            }
            from = row / g.npairs * g.T + p / g.k;
        }
        if (SRC == kScatter) {
            base[j] = row / g.T * g.npairs;
            inv[j] = g.inv + row * g.k;
            bool bad = false;
            if (live[j])
                for (int i = sub; i < g.k; i += lanes) bad |= (uint64_t)__ldg(inv[j] + i) >= (uint64_t)g.npairs;
            if (__ballot_sync(0xffffffffu, bad) & mine) {
                if (sub == 0) set_error(g.hdr, TOPO_ESTATE);
                live[j] = false;
            }
        }
        src[j] = g.x + ((live[j] ? from : 0) * (SRC == kSwiglu ? 2 : 1) * g.nv + sub) * 2;
    }
    Groups<SRC, kN> in_regs;
    in_regs.load(g.nv, [&](int j) { return src[j]; }, [&](int j) { return live[j] && sub < g.nv; },
                 [&](int j) { return __any_sync(0xffffffffu, live[j]) != 0; });
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        if (!__any_sync(0xffffffffu, live[j])) continue;
        const int64_t row = row0 + j * apart;
        float v[16];
        in_regs.get(j, v);
        const uint32_t am = in_regs.amax(j);
        int n = 0;
        if (NV) {
            uint32_t m = am < kInf ? am : finite_bits(v);
            for (int d = lanes >> 1; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
            n = least_power(m, 0x280000u, 11);
        }
        uint32_t sb = to_block<NV>(v, am, n);
        constexpr bool kHalf = NV && SRC != kSwiglu;
        const uint2 q = make_uint2(e2m1x8<kHalf>(v), e2m1x8<kHalf>(v + 8));
        // sixteen blocks' scales on the first of their lanes; those past the row's lanes are 1
        uint32_t w[4];
        const uint32_t s1 = __shfl_down_sync(0xffffffffu, sb, kLanes / 4);
        sb |= (kLanes / 4 < lanes ? s1 : kOne) << 8;
        const uint32_t s2 = __shfl_down_sync(0xffffffffu, sb, kLanes / 2);
        sb |= (kLanes / 2 < lanes ? s2 : kOne * 0x101u) << 16;
        w[0] = sb;
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const uint32_t si = __shfl_down_sync(0xffffffffu, sb, i * kLanes);
            w[i] = i * kLanes < lanes ? si : kOne * 0x1010101u;
        }
        const uint4 word = make_uint4(w[0], w[1], w[2], w[3]);
        const int at = sub / kLanes * 4;
        const bool first = sub % (4 * kLanes) == 0 && at < g.pitch;
        if (!live[j]) continue;
        if (SRC == kScatter) {
            for (int i = 0; i < g.k; ++i) {
                const int64_t r = base[j] + __ldg(inv[j] + i);
                if (sub < g.nv) g.q[r * g.nv + sub] = q;
                if (first) *reinterpret_cast<uint4 *>(g.scale + r * g.pitch + at) = word;
                if (NV && sub == 0) g.row_scale[r] = pow2(n);
            }
        } else {
            if (sub < g.nv) g.q[row * g.nv + sub] = q;
            if (first) *reinterpret_cast<uint4 *>(g.scale + row * g.pitch + at) = word;
            if (NV && sub == 0) g.row_scale[row] = pow2(n);
        }
    }
}

// A lane takes 8 neighbouring values (16 bytes out) four times, 256 values apart, so that
// a warp's stores are whole lines and four loads are on their way at once.  The values and
// codes are one run without gaps, whatever the rows' length: 131072 x 128 7.1 us of MX and
// 6.5 of NV (6.7 TB/s), against 18.2 by rows; 131072 x 7168 336 and 343 us, as by rows.
template <bool NV>
__global__ void __launch_bounds__(256)
k_micro_values(const uint32_t *__restrict__ q, const uint8_t *__restrict__ scale, const float *__restrict__ row_scale, uint4 *out,
               int64_t total, int n8, int pitch) {
    pdl_trigger();
    pdl_wait();
    const int64_t e0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * 128, row0 = e0 / n8;
    if (e0 >= total) return;
    const uint32_t c0 = (uint32_t)(e0 - row0 * n8) + (threadIdx.x & 31);
    const int64_t e = e0 + (threadIdx.x & 31);
    uint32_t w[4], sb[4];
    float g[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t down = (c0 + 32 * j) / (uint32_t)n8, c = c0 + 32 * j - down * n8;
        const int64_t row = row0 + down;
        const bool in = e + 32 * j < total;
        w[j] = in ? __ldcs(q + e + 32 * j) : 0u;
        sb[j] = in ? __ldg(scale + row * pitch + (NV ? c >> 1 : c >> 2)) : 0u;
        g[j] = NV && in ? __ldg(row_scale + row) : 1.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (e + 32 * j >= total) break;
        float s;
        if (NV) s = (sb[j] & 0x7fu) == 0x7fu ? __uint_as_float(0x7fffffffu) : e4m3_value(sb[j]) * g[j];
        else s = sb[j] == 255u ? __uint_as_float(0x7fffffffu) : sb[j] == 0u ? __uint_as_float(0x400000u) : pow2((int)sb[j] - 127);
        uint32_t f[4], o[4];
        asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
            " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
            : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
            : "r"(w[j]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&f[i]));
            const __nv_bfloat162 b = __floats2bfloat162_rn(p.x * s, p.y * s);
            o[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        __stcs(out + e + 32 * j, make_uint4(o[0], o[1], o[2], o[3]));
    }
}

template <int SRC, bool NV, int N>
cudaError_t run_wide(MicroArgs a, cudaStream_t st) {
    a.log_w = 0;
    while (a.log_w < 3 && (N * 32) << a.log_w < a.nv) ++a.log_w;
    const int64_t warps = a.rows << a.log_w;
    return launch_pdl(k_micro_rows<SRC, NV, N>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, a);
}

template <int SRC, bool NV>
cudaError_t run_rows(MicroArgs a, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    // By token, four rows of 17 to 32 groups to a warp leave too few warps that write: 16384
    // tokens, k = 8, H = 288 to NV 24.7 us so, 22.6 by k_micro_rows.
    if (a.nv <= (SRC == kScatter ? 16 : 32)) {
        a.log_l = 1;
        while (1 << a.log_l < a.nv) ++a.log_l;
        const int64_t per = 8 * (kGroups<SRC> * (32 >> a.log_l));   // a CTA's rows
        return launch_pdl(k_micro_narrow<SRC, NV>, dim3((unsigned)((a.rows + per - 1) / per)), dim3(256), 0, st, a);
    }
    if constexpr (SRC == kSwiglu) {
        // Three groups to a lane leave fewer lanes without work in rows of, say, 65 to 96
        // groups: 131072 x 1408 to MX 142 us and to NV 166, against 178 and 225 of two; 2560 270
        // and 333 of three.  With all lanes at work two are the faster (above).
        int w = 64;                                              // groups that one, two, four or eight warps take two to a lane
        while (w < 512 && w < a.nv) w *= 2;
        if (w > 64 && a.nv <= w / 4 * 3) return run_wide<SRC, NV, 3>(a, st);
    }
    return run_wide<SRC, NV, kGroups<SRC>>(a, st);
}

template <int SRC>
cudaError_t run_fmt(const MicroArgs &a, int fmt, cudaStream_t st) {
    return fmt == TOPO_FMT_NV ? run_rows<SRC, true>(a, st) : run_rows<SRC, false>(a, st);
}

MicroArgs row_args(const uint16_t *x, int C, int fmt, uint8_t *q, uint8_t *scale, float *row_scale) {
    MicroArgs a = {};
    a.x = reinterpret_cast<const uint4 *>(x);
    a.q = reinterpret_cast<uint2 *>(q);
    a.scale = scale;
    a.row_scale = row_scale;
    a.nv = C / 16;
    a.pitch = (int)micro_pitch(C, fmt);
    return a;
}

}  // namespace

cudaError_t launch_quantize_rows_micro(int64_t rows, int C, int fmt, const uint16_t *x, uint8_t *q, uint8_t *scale,
                                       float *row_scale, bool swiglu, cudaStream_t st) {
    MicroArgs a = row_args(x, C, fmt, q, scale, row_scale);
    a.rows = rows;
    return swiglu ? run_fmt<kSwiglu>(a, fmt, st) : run_fmt<kPlain>(a, fmt, st);
}

cudaError_t launch_permute_quantize_micro(const Geo &g, int H, int fmt, const uint16_t *x, const int32_t *sorted, uint8_t *q,
                                          uint8_t *scale, float *row_scale, void *ws, cudaStream_t st) {
    MicroArgs a = row_args(x, H, fmt, q, scale, row_scale);
    a.hdr = ws_at<WsHeader>(ws, 0);
    a.npairs = g.npairs;
    a.T = g.T;
    a.k = g.k;
    if ((int64_t)g.L * g.T * H * 2 <= kGatherBytes) {
        a.rows = (int64_t)g.L * g.npairs;
        a.inv = sorted;
        return run_fmt<kGather>(a, fmt, st);
    }
    cudaError_t e;
    if ((e = launch_invert(g, sorted, ws, st)) != cudaSuccess) return e;
    a.rows = (int64_t)g.L * g.T;
    a.inv = ws_at<int32_t>(ws, g.off_pack_inv);
    return run_fmt<kScatter>(a, fmt, st);
}

cudaError_t launch_dequantize_micro(int64_t rows, int C, int fmt, const uint8_t *q, const uint8_t *scale, const float *row_scale,
                                    uint16_t *out, cudaStream_t st) {
    const int n8 = C / 8, pitch = (int)micro_pitch(C, fmt);
    const int64_t total = rows * n8;
    if (total == 0) return cudaSuccess;
    const dim3 grid((unsigned)((total + 1023) / 1024));
    const uint32_t *qv = reinterpret_cast<const uint32_t *>(q);
    uint4 *ov = reinterpret_cast<uint4 *>(out);
    if (fmt == TOPO_FMT_NV)
        return launch_pdl(k_micro_values<true>, grid, dim3(256), 0, st, qv, scale, row_scale, ov, total, n8, pitch);
    return launch_pdl(k_micro_values<false>, grid, dim3(256), 0, st, qv, scale, row_scale, ov, total, n8, pitch);
}

}  // namespace topo
