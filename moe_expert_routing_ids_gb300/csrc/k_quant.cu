// 8-bit operands of the experts' products: e4m3 values with one scale for each
// block of 128 values along the contraction.
//
// A block's scale is the smallest power of two s with amax <= 448 s (exponent
// at least -126; 1 for a block of zeros), amax over the block's finite values;
// q = e4m3(v / s), to nearest, ties to even.  Scaling by a power of two is
// exact, so a value is rounded once.  NaN and infinities become NaN.
//
//   k_quant_rows    rows as they are, dispatch rows (token row t to the k
//                   layout positions of its pairs), or the gated activation
//                   silu(g) * u of rows [g | u]
//   k_quant_cols    128-row blocks of a segment down each column, transposed:
//                   the operands of the weight gradient
//   k_quant_weight  128 x 128 blocks of the experts' weights, and their
//                   transpose (the operand of the input gradient)
//   k_swiglu_grad   gradient of silu(g) * u
//
// A lane takes 16 consecutive values (32 bytes in, 16 bytes out), 8 lanes share a
// block.  Measured: dispatch of 65536 tokens, k = 8, H = 7168: 781 us, 6.2 TB/s,
// 91 percent of a copy's rate, and 5 us for the inverse permutation;
// activation of 131072 rows, I = 2048: 285 us, bound by issue (75 percent of the
// slots: exp and two rounded operations and a rounded division a value; the bytes
// alone would take 200 us); its gradient 411 us, 6.5 TB/s; columns of 98304 rows x
// 2816 and x 4096: 247 us each on average, 4.2 TB/s, 128 registers and two CTAs an
// SM for the next columns' loads; weights of 64 experts, 2816 x 4096, with their
// transposes 597 us, 4.9 TB/s, without 437; 98304 rows of 4096 195 us, 6.3 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "rows.cuh"

namespace topo {
namespace {

enum { kPlain = 0, kScatter = 1, kSwiglu = 2, kGather = 3 };

// Scale of a block whose largest finite magnitude is amax, and its inverse.
__device__ __forceinline__ float scale_of(float amax, float &inv) {
    const uint32_t u = __float_as_uint(amax);
    int n = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);   // 448 = 1.75 * 2^8
    n = max(n, -126);
    if (u == 0u) n = 0;
    inv = __uint_as_float((uint32_t)(127 - n) << 23);
    return __uint_as_float((uint32_t)(127 + n) << 23);
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// Two e4m3 values, lo in the low byte.
__device__ __forceinline__ uint32_t cvt2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Largest finite magnitude of 16 values; NaN and infinities are made NaN.
__device__ __forceinline__ float amax16(float (&v)[16]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));      // fmaxf drops a NaN
    if (!finite(m)) {
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (finite(v[i])) m = fmaxf(m, fabsf(v[i]));
            else v[i] = __int_as_float(0x7fffffff);
        }
    }
    return m;
}

__device__ __forceinline__ uint4 quant16(const float (&v)[16], float inv) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = cvt2(v[4 * i] * inv, v[4 * i + 1] * inv) | (cvt2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16);
    return make_uint4(q[0], q[1], q[2], q[3]);
}

struct QuantArgs {
    const uint4 *x;          // bf16 rows, two uint4 per 16 values
    const int32_t *inv;      // kScatter: position of each pair; kGather: pair of each position
    uint4 *q;                // e4m3 rows
    float *scale;            // [rows][KB]
    WsHeader *hdr;
    int64_t rows;            // rows over all layers (kGather: output rows)
    int64_t npairs;
    int T, k;                // kScatter, kGather: tokens per layer, copies of a row
    int nv;                  // 16-value groups per (output) row
    int KB;
    int parts, per;          // a row is split over `parts` warps of `per` groups of 32 lanes
};

template <int SRC>
__global__ void __launch_bounds__(256)
k_quant_rows(QuantArgs g) {
    const int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t row = unit / g.parts;
    if (row >= g.rows) return;                                   // whole warp
    const int part = (int)(unit - row * g.parts);
    const int lane = threadIdx.x & 31;
    int pa = 0, pb = 0;
    int64_t base = 0, from = row;
    pdl_trigger();
    pdl_wait();
    if (SRC == kGather) {
        const int64_t l = row / g.npairs;
        const int p = __ldg(g.inv + row);
        if ((uint64_t)p >= (uint64_t)g.npairs) {
            if (lane == 0) set_error(g.hdr, TOPO_ESTATE);
            return;
        }
        from = l * g.T + p / g.k;
    }
    if (SRC == kScatter) {
        base = (row / g.T) * g.npairs;
        const int32_t *iv = g.inv + row * g.k;
        pa = lane < g.k ? __ldg(iv + lane) : 0;
        pb = lane + 32 < g.k ? __ldg(iv + lane + 32) : 0;
        if (!__all_sync(0xffffffffu, (uint64_t)pa < (uint64_t)g.npairs && (uint64_t)pb < (uint64_t)g.npairs)) {
            if (lane == 0) set_error(g.hdr, TOPO_ESTATE);
            return;
        }
    }
    const int end = min(g.nv, (part + 1) * g.per * 32);
    for (int c0 = part * g.per * 32; c0 < end; c0 += 32) {
        const int c = c0 + lane;
        const bool in = c < g.nv;
        float v[16];
        const uint4 z = make_uint4(0, 0, 0, 0);
        if (SRC == kSwiglu) {
            const uint4 *src = g.x + row * (4 * (int64_t)g.nv);
            float u[16];
            unpack16(in ? __ldcs(src + 2 * c) : z, in ? __ldcs(src + 2 * c + 1) : z, v);
            src += 2 * g.nv;
            unpack16(in ? __ldcs(src + 2 * c) : z, in ? __ldcs(src + 2 * c + 1) : z, u);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(__fdiv_rn(v[i], __fadd_rn(1.f, expf(-v[i]))), u[i]);
        } else {
            const uint4 *src = g.x + from * (2 * (int64_t)g.nv);
            if (SRC == kGather) unpack16(in ? __ldg(src + 2 * c) : z, in ? __ldg(src + 2 * c + 1) : z, v);
            else unpack16(in ? __ldcs(src + 2 * c) : z, in ? __ldcs(src + 2 * c + 1) : z, v);
        }
        float m = amax16(v);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float iv;
        const float s = scale_of(m, iv);
        const uint4 q = quant16(v, iv);
        if (SRC == kScatter) {
            for (int j = 0; j < g.k; ++j) {
                const int a = __shfl_sync(0xffffffffu, pa, j & 31), b = __shfl_sync(0xffffffffu, pb, j & 31);
                const int64_t r = base + (j < 32 ? a : b);
                if (in) {
                    g.q[r * g.nv + c] = q;
                    if ((lane & 7) == 0) g.scale[r * g.KB + (c >> 3)] = s;
                }
            }
        } else if (in) {
            g.q[row * g.nv + c] = q;
            if ((lane & 7) == 0) g.scale[row * g.KB + (c >> 3)] = s;
        }
    }
}

// The sigmoid by the approximate exp and division: within 1e-5 of itself, 1/200 of the
// bf16 rounding that follows, and 0 for g below -87, where it is below 2^-125.  The
// bytes of the forward pass are not formed here.
__global__ void __launch_bounds__(256)
k_swiglu_grad(const uint4 *__restrict__ h, const uint4 *__restrict__ dy, uint4 *dh, int64_t n, int nv) {
    pdl_trigger();
    pdl_wait();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / nv;
        const int64_t at = row * nv * 2 + (i - row * nv);
        const uint4 a = __ldcs(h + at), b = __ldcs(h + at + nv), d = __ldcs(dy + i);
        const uint32_t qa[4] = {a.x, a.y, a.z, a.w}, qb[4] = {b.x, b.y, b.z, b.w}, qd[4] = {d.x, d.y, d.z, d.w};
        uint32_t rg[4], ru[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float og[2], ou[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float gg = __uint_as_float(e ? qa[j] & 0xffff0000u : qa[j] << 16);
                const float u = __uint_as_float(e ? qb[j] & 0xffff0000u : qb[j] << 16);
                const float y = __uint_as_float(e ? qd[j] & 0xffff0000u : qd[j] << 16);
                const float s = __fdividef(1.f, 1.f + __expf(-gg));
                og[e] = y * u * s * (1.f + gg * (1.f - s));
                ou[e] = y * gg * s;
            }
            const __nv_bfloat162 x = __floats2bfloat162_rn(og[0], og[1]), z = __floats2bfloat162_rn(ou[0], ou[1]);
            rg[j] = *reinterpret_cast<const uint32_t *>(&x);
            ru[j] = *reinterpret_cast<const uint32_t *>(&z);
        }
        __stcs(dh + at, make_uint4(rg[0], rg[1], rg[2], rg[3]));
        __stcs(dh + at + nv, make_uint4(ru[0], ru[1], ru[2], ru[3]));
    }
}

// Two bf16 magnitudes at a time.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// 16 rows of one column (scaled bf16, in the low or high half of their words) as
// 16 e4m3 bytes.
template <bool HI>
__device__ __forceinline__ uint4 quant_col(const uint32_t (&v)[16]) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(HI ? v[4 * i + j] & 0xffff0000u : v[4 * i + j] << 16);
        q[i] = cvt2(f[0], f[1]) | (cvt2(f[2], f[3]) << 16);
    }
    return make_uint4(q[0], q[1], q[2], q[3]);
}

// Values of a word that are not finite made NaN.
__device__ __forceinline__ uint32_t nan2(uint32_t v) {
    if ((v & 0x7fffu) >= 0x7f80u) v |= 0x7fffu;
    if ((v >> 16 & 0x7fffu) >= 0x7f80u) v |= 0x7fff0000u;
    return v;
}

// Two bf16 values times powers of two: exact, but for results that e4m3 rounds to
// zero anyway.
__device__ __forceinline__ uint32_t mul_bf2(uint32_t v, uint32_t by) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&by));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// A CTA takes one row block and 128 columns at a time, the next ones' loads on
// their way meanwhile: warp w holds rows 16 w .. 16 w + 15, lane l columns 4 l ..
// 4 l + 3; 16 rows of a column are one 16-byte piece of the transposed row.  The
// pieces pass through shared memory (piece index XOR the lane, so that 8 lanes
// hit 8 bank groups) to leave in whole 128-byte rows.
__global__ void __launch_bounds__(256, 2)
k_quant_cols(const uint16_t *__restrict__ x, const int32_t *__restrict__ seg_off, uint8_t *q, float *scale, WsHeader *hdr,
             int nseg, int64_t rows, int C, int64_t cap) {
    __shared__ uint4 tile[2][128 * 8];
    __shared__ uint2 wmax[2][8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x;
    pdl_trigger();
    pdl_wait();
    // the segment of padded block b
    int seg = -1, r0 = 0, nrow = 0, run = 0;
    for (int i0 = 0; i0 < nseg && seg < 0; i0 += 32) {
        const int i = i0 + lane;
        int n = 0, a = 0, e = 0;
        if (i < nseg) {
            a = __ldg(seg_off + i);
            e = __ldg(seg_off + i + 1);
            if (a < 0 || e < a || e > rows) set_error(hdr, TOPO_ESTATE);
            else n = (e - a + 127) / 128;
        }
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        const int lo = run + s - n;
        const unsigned hit = __ballot_sync(0xffffffffu, b >= lo && b < lo + n);
        if (hit) {
            const int w = __ffs(hit) - 1;
            seg = i0 + w;
            r0 = __shfl_sync(0xffffffffu, a + (b - lo) * 128, w);
            nrow = min(128, __shfl_sync(0xffffffffu, e, w) - r0);
        }
        run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (seg < 0) return;                                          // past the last segment's blocks
    const uint16_t *src = x + (int64_t)(r0 + 16 * warp) * C + 4 * lane;
    uint2 nx[16];
    auto load = [&](int c0) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            nx[r] = c0 + 4 * lane < C && 16 * warp + r < nrow
                        ? __ldcs(reinterpret_cast<const uint2 *>(src + (int64_t)r * C + c0)) : make_uint2(0, 0);
    };
    int c0 = blockIdx.y * 128, s = 0;
    if (c0 < C) load(c0);
    for (; c0 < C; c0 += gridDim.y * 128, s ^= 1) {
        uint32_t v0[16], v1[16];
        uint2 m = make_uint2(0, 0);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            v0[r] = nx[r].x;
            v1[r] = nx[r].y;
            m.x = max2(m.x, v0[r] & 0x7fff7fffu);
            m.y = max2(m.y, v1[r] & 0x7fff7fffu);
        }
        // some value of this warp's column is not finite: taken again without those
        const bool odd = (m.x & 0x7fffu) >= 0x7f80u || (m.x >> 16) >= 0x7f80u || (m.y & 0x7fffu) >= 0x7f80u || (m.y >> 16) >= 0x7f80u;
        if (odd) {
            m = make_uint2(0, 0);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                uint32_t a = v0[r] & 0x7fff7fffu, c = v1[r] & 0x7fff7fffu;
                if ((a & 0x7fffu) >= 0x7f80u) a &= 0xffff0000u;
                if ((a >> 16) >= 0x7f80u) a &= 0xffffu;
                if ((c & 0x7fffu) >= 0x7f80u) c &= 0xffff0000u;
                if ((c >> 16) >= 0x7f80u) c &= 0xffffu;
                m.x = max2(m.x, a);
                m.y = max2(m.y, c);
                v0[r] = nan2(v0[r]);
                v1[r] = nan2(v1[r]);
            }
        }
        if (c0 + (int)gridDim.y * 128 < C) load(c0 + gridDim.y * 128);
        wmax[s][warp][lane] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const uint2 o = wmax[s][w][lane];
            m.x = max2(m.x, o.x);
            m.y = max2(m.y, o.y);
        }
        const int c = c0 + 4 * lane;
        float iv[4], sc[4];
        sc[0] = scale_of(__uint_as_float(m.x << 16), iv[0]);
        sc[1] = scale_of(__uint_as_float(m.x & 0xffff0000u), iv[1]);
        sc[2] = scale_of(__uint_as_float(m.y << 16), iv[2]);
        sc[3] = scale_of(__uint_as_float(m.y & 0xffff0000u), iv[3]);
        uint4 *t = tile[s] + 32 * lane + (warp ^ (lane & 7));
        const uint32_t b0 = (__float_as_uint(iv[0]) >> 16) | (__float_as_uint(iv[1]) & 0xffff0000u);
        const uint32_t b1 = (__float_as_uint(iv[2]) >> 16) | (__float_as_uint(iv[3]) & 0xffff0000u);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            v0[r] = mul_bf2(v0[r], b0);
            v1[r] = mul_bf2(v1[r], b1);
        }
        t[0] = quant_col<false>(v0);
        t[8] = quant_col<true>(v0);
        t[16] = quant_col<false>(v1);
        t[24] = quant_col<true>(v1);
        if (warp == 0 && c < C) {
#pragma unroll
            for (int j = 0; j < 4; ++j) scale[(int64_t)b * C + c + j] = sc[j];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = i * 256 + threadIdx.x, cc = e >> 3, ch = e & 7;
            if (c0 + cc < C)
                *reinterpret_cast<uint4 *>(q + (int64_t)(c0 + cc) * cap + (int64_t)b * 128 + 16 * ch) =
                    tile[s][cc * 8 + (ch ^ ((cc >> 2) & 7))];
        }
    }
}

// One CTA per 128 x 128 block of a weight matrix [N][K].
__global__ void __launch_bounds__(256)
k_quant_weight(const uint16_t *__restrict__ w, uint8_t *q, float *scale, uint8_t *qt, float *scale_t, int N, int K) {
    __shared__ float red[8];
    __shared__ uint8_t tile[128][132];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int KB = (K + 127) / 128, NB = (N + 127) / 128;
    const int kb = blockIdx.x, nb = blockIdx.y;
    const int64_t base = (int64_t)blockIdx.z * N * K;
    const int k = kb * 128 + 4 * lane;
    uint2 v[16];
    float m = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int n = nb * 128 + 16 * warp + r;
        v[r] = n < N && k < K ? __ldcs(reinterpret_cast<const uint2 *>(w + base + (int64_t)n * K + k)) : make_uint2(0, 0);
        const uint32_t p[4] = {v[r].x << 16, v[r].x & 0xffff0000u, v[r].y << 16, v[r].y & 0xffff0000u};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float f = __uint_as_float(p[j]);
            if (finite(f)) m = fmaxf(m, fabsf(f));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
    float iv;
    const float s = scale_of(m, iv);
    if (threadIdx.x == 0) {
        scale[((int64_t)blockIdx.z * NB + nb) * KB + kb] = s;
        if (scale_t) scale_t[((int64_t)blockIdx.z * KB + kb) * NB + nb] = s;
    }
    const float nan = __int_as_float(0x7fffffff);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int n = nb * 128 + 16 * warp + r;
        float f[4] = {__uint_as_float(v[r].x << 16), __uint_as_float(v[r].x & 0xffff0000u),
                      __uint_as_float(v[r].y << 16), __uint_as_float(v[r].y & 0xffff0000u)};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (!finite(f[j])) f[j] = nan;
        const uint32_t e = cvt2(f[0] * iv, f[1] * iv) | (cvt2(f[2] * iv, f[3] * iv) << 16);
        if (n < N && k < K) *reinterpret_cast<uint32_t *>(q + base + (int64_t)n * K + k) = e;
        *reinterpret_cast<uint32_t *>(&tile[16 * warp + r][4 * lane]) = e;
    }
    if (!qt) return;
    __syncthreads();
    const int n = nb * 128 + 4 * lane;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int kk = 16 * warp + r;
        uint32_t e = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) e |= (uint32_t)tile[4 * lane + j][kk] << (8 * j);
        if (kb * 128 + kk < K && n < N) *reinterpret_cast<uint32_t *>(qt + base + (int64_t)(kb * 128 + kk) * N + n) = e;
    }
}

template <int SRC>
cudaError_t run_rows(QuantArgs a, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    const int chunks = (a.nv + 31) / 32;
    // few rows: a row's 512-value chunks go to warps of their own
    a.per = a.rows * chunks <= 152 * 64 ? 1 : chunks;
    a.parts = (chunks + a.per - 1) / a.per;
    const int64_t units = a.rows * a.parts;
    return launch_pdl(k_quant_rows<SRC>, dim3((unsigned)((units + 7) / 8)), dim3(256), 0, st, a);
}

}  // namespace

cudaError_t launch_quantize_rows(int64_t rows, int C, const uint16_t *x, uint8_t *q, float *scale, bool swiglu,
                                 cudaStream_t st) {
    QuantArgs a = {};
    a.x = reinterpret_cast<const uint4 *>(x);
    a.q = reinterpret_cast<uint4 *>(q);
    a.scale = scale;
    a.rows = rows;
    a.nv = C / 16;
    a.KB = (C + 127) / 128;
    return swiglu ? run_rows<kSwiglu>(a, st) : run_rows<kPlain>(a, st);
}

cudaError_t launch_permute_quantize(const Geo &g, int H, const uint16_t *x, const int32_t *sorted, uint8_t *q, float *scale,
                                    void *ws, cudaStream_t st) {
    QuantArgs a = {};
    a.x = reinterpret_cast<const uint4 *>(x);
    a.q = reinterpret_cast<uint4 *>(q);
    a.scale = scale;
    a.hdr = ws_at<WsHeader>(ws, 0);
    a.npairs = g.npairs;
    a.T = g.T;
    a.k = g.k;
    a.nv = H / 16;
    a.KB = (H + 127) / 128;
    if ((int64_t)g.L * g.T * H * 2 <= kGatherBytes) {
        a.rows = (int64_t)g.L * g.npairs;
        a.inv = sorted;
        return run_rows<kGather>(a, st);
    }
    cudaError_t e;
    if ((e = launch_invert(g, sorted, ws, st)) != cudaSuccess) return e;
    a.rows = (int64_t)g.L * g.T;
    a.inv = ws_at<int32_t>(ws, g.off_pack_inv);
    return run_rows<kScatter>(a, st);
}

cudaError_t launch_quantize_cols(int nseg, int64_t rows, int C, const uint16_t *x, const int32_t *seg_off, int64_t cap,
                                 uint8_t *q, float *scale, void *ws, cudaStream_t st) {
    const int64_t blocks = cap / 128;
    const int cb = (C + 127) / 128;
    // two CTAs to an SM run together; finding the row block's segment costs a CTA two
    // round trips to memory, so it takes several column groups where there are
    // enough CTAs: at least 8 / 16 / 24 / 40 to an SM, 98304 rows x 2816 and x 4096:
    // 267 / 254 / 247 / 247 us each on average
    int64_t split = (152 * 24 + blocks - 1) / blocks;
    if (split > cb) split = cb;
    return launch_pdl(k_quant_cols, dim3((unsigned)blocks, (unsigned)split), dim3(256), 0, st, x, seg_off, q, scale,
                      ws_at<WsHeader>(ws, 0), nseg, rows, C, cap);
}

cudaError_t launch_quantize_weight(int n_w, int N, int K, const uint16_t *w, uint8_t *q, float *scale, uint8_t *qt,
                                   float *scale_t, cudaStream_t st) {
    const unsigned KB = (unsigned)((K + 127) / 128), NB = (unsigned)((N + 127) / 128);
    for (int z = 0; z < n_w; z += 65535) {
        const int n = n_w - z < 65535 ? n_w - z : 65535;
        const int64_t o = (int64_t)z * N * K, os = (int64_t)z * NB * KB;
        k_quant_weight<<<dim3(KB, NB, (unsigned)n), 256, 0, st>>>(w + o, q + o, scale + os, qt ? qt + o : nullptr,
                                                                  scale_t ? scale_t + os : nullptr, N, K);
    }
    return cudaGetLastError();
}

cudaError_t launch_swiglu_grad(int64_t rows, int I, const uint16_t *h, const uint16_t *dy, uint16_t *dh, cudaStream_t st) {
    const int nv = I / 8;
    const int64_t n = rows * nv;
    if (n == 0) return cudaSuccess;
    const int64_t want = (n + 255) / 256;
    return launch_pdl(k_swiglu_grad, dim3((unsigned)(want < 152 * 32 ? want : 152 * 32)), dim3(256), 0, st,
                      reinterpret_cast<const uint4 *>(h), reinterpret_cast<const uint4 *>(dy), reinterpret_cast<uint4 *>(dh), n, nv);
}

}  // namespace topo
