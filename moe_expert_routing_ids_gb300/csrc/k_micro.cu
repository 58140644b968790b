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
// scale NaN.  Division by a power of two is exact; the quotient by an e4m3 scale is
// corrected by its residual (Markstein), so that a quotient on the border between
// two values of e2m1, the only place where a last bit counts, comes out exactly.
//
//   k_micro_rows     rows as they are, dispatch rows (by position, or token row t to the
//                    k layout positions of its pairs), or the gated activation
//                    silu(g) * u of rows [g | u]
//   k_micro_values   the bf16 values that such rows stand for
//
// A lane takes 16 consecutive values (32 bytes in, 8 bytes out): a block of NV, half
// a block of MX.
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

// Eight values in 4 bits, the first in the lowest.
__device__ __forceinline__ uint32_t e2m1x8(const float *v) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
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
    int parts, per;          // a row is split over `parts` warps of `per` groups of 32 lanes
    int keep;                // NV, kSwiglu: a row's values pass through shared memory
};

// Bits of the largest magnitude of 16 values (as NaN > infinity > finite values), and of
// the largest finite one where that is neither.
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[16]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}
__device__ __forceinline__ uint32_t finite_bits(const float (&v)[16]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
        if (u < kInf) m = max(m, u);
    }
    return m;
}

// Group c of a source row, zeros past its end.
template <int SRC>
__device__ __forceinline__ void load16(const MicroArgs &g, int64_t from, int c, float (&v)[16]) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    const bool in = c < g.nv;
    if (SRC == kSwiglu) {
        const uint4 *src = g.x + from * (4 * (int64_t)g.nv);
        float u[16];
        unpack16(in ? __ldcs(src + 2 * c) : z, in ? __ldcs(src + 2 * c + 1) : z, v);
        src += 2 * g.nv;
        unpack16(in ? __ldcs(src + 2 * c) : z, in ? __ldcs(src + 2 * c + 1) : z, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(__fdiv_rn(v[i], __fadd_rn(1.f, expf(-v[i]))), u[i]);
    } else {
        const uint4 *src = g.x + from * (2 * (int64_t)g.nv);
        unpack16(in ? __ldg(src + 2 * c) : z, in ? __ldg(src + 2 * c + 1) : z, v);
    }
}

template <int SRC, bool NV>
__global__ void __launch_bounds__(256)
k_micro_rows(MicroArgs g) {
    extern __shared__ float kept[];                              // keep: a row of each warp
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
    float *mine = kept + (threadIdx.x >> 5) * ((g.nv + 31) / 32 * 512);
    float ginv = 1.f;
    if (NV) {
        // the whole row's largest finite magnitude first
        uint32_t m = 0;
        for (int c = lane; c < g.nv; c += 32) {
            float v[16];
            load16<SRC>(g, from, c, v);
            const uint32_t a = amax_bits(v);
            m = max(m, a < kInf ? a : finite_bits(v));
            if (SRC == kSwiglu && g.keep)
#pragma unroll
                for (int i = 0; i < 4; ++i)                      // piece i of each lane side by side
                    *reinterpret_cast<float4 *>(mine + (c >> 5) * 512 + i * 128 + 4 * lane) =
                        make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        const int n = least_power(m, 0x280000u, 11);             // 6 * 448 = 1.3125 * 2^11
        ginv = pow2(-n);
        if (SRC == kScatter && part == 0) {
            if (lane < g.k) g.row_scale[base + pa] = pow2(n);
            if (lane + 32 < g.k) g.row_scale[base + pb] = pow2(n);
        } else if (lane == 0 && part == 0) {
            g.row_scale[row] = pow2(n);
        }
    }
    const int end = min((g.nv + 31) & ~31, (part + 1) * g.per * 32);
    for (int c0 = part * g.per * 32; c0 < end; c0 += 32) {
        const int c = c0 + lane;
        const bool in = c < g.nv;
        float v[16];
        if (NV && SRC == kSwiglu && g.keep) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = in ? *reinterpret_cast<const float4 *>(mine + (c >> 5) * 512 + i * 128 + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[4 * i] = f.x;
                v[4 * i + 1] = f.y;
                v[4 * i + 2] = f.z;
                v[4 * i + 3] = f.w;
            }
        } else {
            load16<SRC>(g, from, c, v);
        }
        uint32_t m = amax_bits(v), sb;
        if (NV) {
            const float t = __uint_as_float(m) * ginv;           // at most 2688
            uint16_t b;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.f), "f"(t * (1.f / 6.f)));
            sb = b;
            float s = e4m3_value(sb);
            if (6.f * s < t) s = e4m3_value(++sb);               // rounded down: the next one
            if (m == 0u) s = 1.f, sb = 0x38u;
            const float si = __frcp_rn(s);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float y = v[i] * ginv, q0 = y * si;
                v[i] = __fmaf_rn(__fmaf_rn(-q0, s, y), si, q0);
            }
            if (m >= kInf) sb = 0x7fu;
        } else {
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            const int n = m < kInf ? least_power(m, 0x400000u, 2) : 0;   // 6 = 1.5 * 2^2
            const float inv = pow2(-n);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= inv;
            sb = m < kInf ? (uint32_t)(127 + n) : 255u;
        }
        const uint2 q = make_uint2(e2m1x8(v), e2m1x8(v + 8));
        // four blocks' scales to a word, on the first of their lanes; bytes past the last
        // block hold 1
        constexpr int kLanes = NV ? 4 : 8;                       // lanes of a word
        sb |= __shfl_down_sync(0xffffffffu, sb, kLanes / 4) << 8;
        sb |= __shfl_down_sync(0xffffffffu, sb, kLanes / 2) << 16;
        const int at = (c0 + lane) / kLanes * 4;
        const bool word = lane % kLanes == 0 && at < g.pitch;
        if (SRC == kScatter) {
            for (int j = 0; j < g.k; ++j) {
                const int a = __shfl_sync(0xffffffffu, pa, j & 31), b = __shfl_sync(0xffffffffu, pb, j & 31);
                const int64_t r = base + (j < 32 ? a : b);
                if (in) g.q[r * g.nv + c] = q;
                if (word) *reinterpret_cast<uint32_t *>(g.scale + r * g.pitch + at) = sb;
            }
        } else {
            if (in) g.q[row * g.nv + c] = q;
            if (word) *reinterpret_cast<uint32_t *>(g.scale + row * g.pitch + at) = sb;
        }
    }
}

// A warp takes 512 values of a row.
template <bool NV>
__global__ void __launch_bounds__(256)
k_micro_values(const uint2 *__restrict__ q, const uint8_t *__restrict__ scale, const float *__restrict__ row_scale, uint4 *out,
               int64_t units, int nv, int pitch) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, chunks = (nv + 31) / 32;
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * 8) {
        const int64_t row = u / chunks;
        const int c = (int)(u - row * chunks) * 32 + lane;
        if (c >= nv) continue;
        const uint2 w = __ldcs(q + row * nv + c);
        const uint32_t sb = __ldg(scale + row * pitch + (NV ? c : c >> 1));
        float s;
        if (NV) s = (sb & 0x7fu) == 0x7fu ? __uint_as_float(0x7fffffffu) : e4m3_value(sb) * __ldg(row_scale + row);
        else s = sb == 255u ? __uint_as_float(0x7fffffffu) : sb == 0u ? __uint_as_float(0x400000u) : pow2((int)sb - 127);
        uint32_t o[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t f[4];
            asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
                " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
                : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
                : "r"(h ? w.y : w.x));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&f[i]));
                const __nv_bfloat162 b = __floats2bfloat162_rn(p.x * s, p.y * s);
                o[4 * h + i] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
        uint4 *dst = out + (row * nv + c) * 2;
        __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
    }
}

template <int SRC, bool NV>
cudaError_t run_rows(MicroArgs a, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    const int chunks = (a.nv + 31) / 32;
    // few rows: a row's 512-value chunks go to warps of their own
    a.per = a.rows * chunks <= 152 * 64 ? 1 : chunks;
    a.parts = (chunks + a.per - 1) / a.per;
    const int64_t units = a.rows * a.parts;
    size_t smem = 0;
    if (NV && SRC == kSwiglu && a.parts == 1 && chunks <= 13) {  // 8 warps' rows of 512 float32 a chunk
        a.keep = 1;
        smem = (size_t)8 * chunks * 2048;
        const cudaError_t e = ensure_smem((const void *)k_micro_rows<SRC, NV>, smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(k_micro_rows<SRC, NV>, dim3((unsigned)((units + 7) / 8)), dim3(256), smem, st, a);
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
    const int nv = C / 16, pitch = (int)micro_pitch(C, fmt);
    const int64_t units = rows * ((nv + 31) / 32);
    if (units == 0) return cudaSuccess;
    const int64_t want = (units + 7) / 8;
    const dim3 grid((unsigned)(want < 152 * 32 ? want : 152 * 32));
    const uint2 *qv = reinterpret_cast<const uint2 *>(q);
    uint4 *ov = reinterpret_cast<uint4 *>(out);
    if (fmt == TOPO_FMT_NV)
        return launch_pdl(k_micro_values<true>, grid, dim3(256), 0, st, qv, scale, row_scale, ov, units, nv, pitch);
    return launch_pdl(k_micro_values<false>, grid, dim3(256), 0, st, qv, scale, row_scale, ov, units, nv, pitch);
}

}  // namespace topo
