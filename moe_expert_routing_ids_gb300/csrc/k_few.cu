// The experts applied to a few tokens:
//   out[t] = sum_j w[t][j] * W_down[e] (silu(g) * u),  [g | u] = W_up[e] x[t],  e = ids[t][j]
//
// The weights of the experts in use are read once and are all the traffic; a token's
// products are next to nothing.  Two kernels, up and down, one CTA to an SM:
//
//   items   a tile of 16 weight rows (8 gate rows and their 8 up rows; 16 rows of
//           W_down) of one expert in use, in the experts' order; a CTA takes an equal
//           share of neighbouring items, its warps one after the other (or, where a CTA
//           has fewer items of an expert than warps, a part of the contraction each)
//   weights each warp streams its rows through its own ring of shared memory, 128 bytes
//           of each row a stage, by cp.async: no warp waits for another
//   product mma.sync m16n8k16 in f16 with float32 sums: weight rows on M, tokens on N.
//           e4m3 and e2m1 are f16 values; scales by 128 and by 32 multiply a block's
//           sum, scales by 16 the f16 weights (6 bits: exact)
//   tokens  as f16 over a power of two for each row (its largest magnitude in
//           [2^14, 2^15)): 11 bits, where bf16 has 8
//   sums    float32 throughout: an expert's outputs for a token go to the workspace, and
//           the warp that brings the last expert's of 16 columns adds them in slot order
//           with their weights, so the result does not depend on who comes last
//
// The down kernel starts while the up kernel runs (its first weights do not depend on
// it) and waits for it before it reads the activations.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"

namespace topo {
namespace {

constexpr int kSms = 152;
constexpr int kMaxWarps = 16;
constexpr int kRowBytes = 128;                    // of a weight row in a stage
constexpr int kSfRow = 16;                        // scale bytes of a row in a stage, at most
constexpr int kStageBytes = 16 * (kRowBytes + kSfRow);
constexpr int kMaxTokens = 8;                     // of one launch, the N of a product
constexpr int kMaxPairs = kMaxTokens * kMaxK;
constexpr int kMaxRows = 16;                      // token rows that a CTA holds
constexpr int kMaxParts = 64;                     // partial tiles that it holds
constexpr int kCounters = (1 << 15) / 16;         // column tiles of the widest H

struct FewArgs {
    const uint16_t *x;          // up: bf16 [T][K]
    const float *act;           // down: [T * k][K]
    const int32_t *ids;         // [T][k]
    const float *weights;       // [T][k]
    const uint8_t *w;           // [E][rows][K]
    const uint8_t *scale;
    const float *row_scale;     // NV
    float *mid;                 // up: act; down: y [T * k][H]
    uint16_t *out;              // down: [T][H]
    int32_t *count;             // [H / 16] experts done
    WsHeader *hdr;
    int T, E, k;
    int K, I, H;                // values contracted; the layer's sizes
    int rows;                   // weight rows of an expert
    int units;                  // tiles of 16 rows of an expert
    int nc;                     // stages of a row
    int64_t pitch;              // 4 bits: scale bytes of a row
    int bpitch;                 // bytes of a token row in shared memory
    int warps, cap_rows, cap_parts;
};

__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// 16 bytes, or zeros
__device__ __forceinline__ void copy_or_zero(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 values as f16.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}
// Eight e2m1 values as f16.
__device__ __forceinline__ void e2m1x8(uint32_t v, uint32_t (&r)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(v));
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Exponent e of a row's factor: largest magnitude (bits) in [2^14, 2^15) after * 2^-e.
__device__ __forceinline__ int row_exp(uint32_t amax) { return max((int)(amax >> 23) - 127 - 14, -126); }
__device__ __forceinline__ float pow2(int n) { return __uint_as_float((uint32_t)(127 + n) << 23); }

// Position of a row's 16-byte piece c in its 128 bytes of a stage: 16-byte reads of two
// rows' four pieces, or 4-byte reads of one piece of eight rows, hit all banks once.
template <int FMT>
__device__ __forceinline__ int piece(int row, int c) {
    return (c ^ (FMT == TOPO_FMT_EIGHT ? (row & 1) << 2 : row & 7)) * 16;
}

// acc += the product of a stage: 16 weight rows, 128 or 256 values, 8 token columns.
// K within a stage is dealt to the lanes in whole pieces, the same for weights and tokens.
template <int FMT>
__device__ __forceinline__ void stage_product(float (&acc)[4], const unsigned char *st, const unsigned char *b, int lane) {
    const int r = lane >> 2, t = lane & 3;
    const unsigned char *sf = st + 16 * kRowBytes;
    if constexpr (FMT == TOPO_FMT_EIGHT) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {                           // 64 values, 16 of them this lane's
            const uint4 v0 = *reinterpret_cast<const uint4 *>(st + r * kRowBytes + piece<FMT>(r, 4 * q + t));
            const uint4 v1 = *reinterpret_cast<const uint4 *>(st + (r + 8) * kRowBytes + piece<FMT>(r, 4 * q + t));
            const uint32_t p0[4] = {v0.x, v0.y, v0.z, v0.w}, p1[4] = {v1.x, v1.y, v1.z, v1.w};
            uint32_t f[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j][0] = e4m3x2(p0[j]);
                f[j][1] = e4m3x2(p1[j]);
                f[j][2] = e4m3x2(p0[j] >> 16);
                f[j][3] = e4m3x2(p1[j] >> 16);
            }
            const uint4 x0 = *reinterpret_cast<const uint4 *>(b + 128 * q + 32 * t);
            const uint4 x1 = *reinterpret_cast<const uint4 *>(b + 128 * q + 32 * t + 16);
            mma16(d, f[0], x0.x, x0.y);
            mma16(d, f[1], x0.z, x0.w);
            mma16(d, f[2], x1.x, x1.y);
            mma16(d, f[3], x1.z, x1.w);
        }
        const float2 s = *reinterpret_cast<const float2 *>(sf);
        acc[0] += d[0] * s.x;
        acc[1] += d[1] * s.x;
        acc[2] += d[2] * s.y;
        acc[3] += d[3] * s.y;
    } else {
        uint32_t s0[4], s1[4];                                  // the scales of rows r and r + 8
        if (FMT == TOPO_FMT_NV) {
            const uint4 a = *reinterpret_cast<const uint4 *>(sf + r * 16), c = *reinterpret_cast<const uint4 *>(sf + (r + 8) * 16);
            s0[0] = a.x, s0[1] = a.y, s0[2] = a.z, s0[3] = a.w;
            s1[0] = c.x, s1[1] = c.y, s1[2] = c.z, s1[3] = c.w;
        } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(sf + r * 16), c = *reinterpret_cast<const uint2 *>(sf + (r + 8) * 16);
            s0[0] = a.x, s0[1] = a.y;
            s1[0] = c.x, s1[1] = c.y;
        }
        const uint32_t pick = t < 2 ? 0x1010u : 0x3232u;        // NV: this lane's of a 32-value piece's two scales
#pragma unroll
        for (int q = 0; q < 8; ++q) {                           // 32 values, 8 of them this lane's
            uint32_t f0[4], f1[4];
            e2m1x8(*reinterpret_cast<const uint32_t *>(st + r * kRowBytes + piece<FMT>(r, q) + 4 * t), f0);
            e2m1x8(*reinterpret_cast<const uint32_t *>(st + (r + 8) * kRowBytes + piece<FMT>(r, q) + 4 * t), f1);
            if (FMT == TOPO_FMT_NV) {
                const uint32_t c0 = __byte_perm(e4m3x2(s0[q >> 1] >> (16 * (q & 1))), 0, pick);
                const uint32_t c1 = __byte_perm(e4m3x2(s1[q >> 1] >> (16 * (q & 1))), 0, pick);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f0[i] = mul2(f0[i], c0);
                    f1[i] = mul2(f1[i], c1);
                }
            }
            const uint32_t a0[4] = {f0[0], f1[0], f0[1], f1[1]}, a1[4] = {f0[2], f1[2], f0[3], f1[3]};
            float m0 = 0.f, m1 = 0.f;
            if (FMT == TOPO_FMT_MX) {                           // 2^(byte - 127), 2^-127 for a byte of 0
                const uint32_t u0 = (s0[q >> 2] >> (8 * (q & 3))) << 23, u1 = (s1[q >> 2] >> (8 * (q & 3))) << 23;
                m0 = __uint_as_float(max(u0 & 0x7f800000u, 0x400000u));
                m1 = __uint_as_float(max(u1 & 0x7f800000u, 0x400000u));
            }
            const uint4 x = *reinterpret_cast<const uint4 *>(b + 64 * q + 16 * t);
            if (FMT == TOPO_FMT_NV) {
                mma16(acc, a0, x.x, x.y);
                mma16(acc, a1, x.z, x.w);
            } else {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma16(d, a0, x.x, x.y);
                mma16(d, a1, x.z, x.w);
                acc[0] += d[0] * m0;
                acc[1] += d[1] * m0;
                acc[2] += d[2] * m1;
                acc[3] += d[3] * m1;
            }
        }
    }
}

// Issues one warp's stages of its items in order, ahead of their use.
template <int FMT, bool DOWN>
struct Feed {
    const unsigned char *src[4];                                // this lane's piece of rows lane / 8 + 4 i
    const unsigned char *sf;                                    // this lane's scales
    int item, chunk, last;                                      // the next stage: its item, stages of it, its end

    // First row of a tile in the expert's weights, from row h of the 16.
    static __device__ __forceinline__ int64_t row_of(const FewArgs &g, int unit, int h) {
        return DOWN ? 16 * unit + h : h < 8 ? 8 * unit + h : g.I + 8 * unit + h - 8;
    }
    __device__ __forceinline__ void begin(const FewArgs &g, int e, int unit, int part, int log_s, int lane) {
        chunk = (part * g.nc) >> log_s;
        last = ((part + 1) * g.nc) >> log_s;
        const int64_t kb = FMT == TOPO_FMT_EIGHT ? g.K : g.K / 2;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            src[i] = g.w + ((int64_t)e * g.rows + row_of(g, unit, (lane >> 3) + 4 * i)) * kb + 16 * (lane & 7);
        if (FMT == TOPO_FMT_EIGHT) {
            // the float32 of a 128 x 128 block: of the gate rows and of the up rows
            const int64_t nb = (g.rows + 127) / 128, at = (int64_t)e * nb + row_of(g, unit, lane & 1 ? 8 : 0) / 128;
            sf = g.scale + at * g.nc * 4;
        } else {
            sf = g.scale + ((int64_t)e * g.rows + row_of(g, unit, lane & 15)) * g.pitch;
        }
    }
    __device__ __forceinline__ void issue(const FewArgs &g, unsigned char *st, int lane) const {
        const int kb = FMT == TOPO_FMT_EIGHT ? g.K : g.K / 2;
        const int64_t at = (int64_t)chunk * kRowBytes;
        const bool in = at + 16 * (lane & 7) < kb;
        const uint32_t dst = smem_at(st);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (lane >> 3) + 4 * i;
            copy_or_zero(dst + row * kRowBytes + piece<FMT>(row, lane & 7), in ? src[i] + at : g.w, in);
        }
        const uint32_t ds = dst + 16 * kRowBytes;
        if (FMT == TOPO_FMT_EIGHT) {
            if (lane < 2) copy_async<4>(ds + 4 * lane, sf + 4 * chunk);
        } else if (lane < 16) {
            if (FMT == TOPO_FMT_NV) copy_async<16>(ds + 16 * lane, sf + 16 * chunk);
            else copy_async<8>(ds + 16 * lane, sf + 8 * chunk);
        }
    }
};

// The largest finite magnitude of eight bf16 values as float32 bits.
__device__ __forceinline__ uint32_t finite_amax(const uint4 &a) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, u[i] & 0x7fff7fffu);
    if ((m >> 16) >= 0x7f80u || (m & 0xffffu) >= 0x7f80u) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = u[i] & 0x7fffu, hi = u[i] >> 16 & 0x7fffu;
            m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
        return m << 16;
    }
    return max(m << 16, m & 0xffff0000u);
}

// A token row of bf16 in shared memory made f16 in its place; the lane's pieces of 8 are
// c0, c0 + dc, ...  Each warp of the CTA calls it, with rows (`on`) or without.
__device__ __forceinline__ void convert_rows(unsigned char *tok, uint32_t *amax, bool on, int c0, int dc, int kpad) {
    uint32_t m = 0;
    if (on)
        for (int c = c0; c < kpad / 8; c += dc) m = max(m, finite_amax(*reinterpret_cast<const uint4 *>(tok + 16 * c)));
    m = __reduce_max_sync(0xffffffffu, m);
    if (on && (threadIdx.x & 31) == 0) atomicMax(amax, m);
    __syncthreads();
    if (!on) return;
    const float mul = pow2(-row_exp(*amax));
    for (int c = c0; c < kpad / 8; c += dc) {
        uint4 *p = reinterpret_cast<uint4 *>(tok + 16 * c);
        const uint4 a = *p;
        uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = pack_f16(__uint_as_float(u[i] << 16) * mul, __uint_as_float(u[i] & 0xffff0000u) * mul);
        *p = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// An activation row as f16 in shared memory, in the same pieces; up to kKeep of them stay
// in registers between the row's largest magnitude and the conversion, more are read twice.
template <int FMT>
__device__ __forceinline__ void load_act(const FewArgs &g, unsigned char *tok, uint32_t *amax, bool on, int row, int pair, int c0,
                                         int dc, int kpad) {
    constexpr int kKeep = 4;
    const float4 *src = reinterpret_cast<const float4 *>(g.act + (int64_t)pair * g.K);
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 v[kKeep][2];
    const int n = on ? (kpad / 8 - c0 + dc - 1) / dc : 0;
    uint32_t m = 0;
    for (int i0 = 0; i0 < n; i0 += kKeep) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int c = c0 + (i0 + i) * dc;
            const bool in = i0 + i < n && c < g.K / 8;
            v[i][0] = in ? __ldcg(src + 2 * c) : z;
            v[i][1] = in ? __ldcg(src + 2 * c + 1) : z;
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const float f[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = __float_as_uint(f[j]) & 0x7fffffffu;
                if (u < 0x7f800000u) m = max(m, u);
            }
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (on && (threadIdx.x & 31) == 0) atomicMax(&amax[row], m);
    __syncthreads();
    if (!on) return;
    const float mul = pow2(-row_exp(amax[row]));
    for (int i0 = 0; i0 < n; i0 += kKeep) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int c = c0 + (i0 + i) * dc;
            if (i0 + i >= n) break;
            if (n > kKeep) {
                v[i][0] = c < g.K / 8 ? __ldcg(src + 2 * c) : z;
                v[i][1] = c < g.K / 8 ? __ldcg(src + 2 * c + 1) : z;
            }
            const float4 a = v[i][0], d = v[i][1];
            *reinterpret_cast<uint4 *>(tok + row * g.bpitch + 16 * c) =
                make_uint4(pack_f16(a.x * mul, a.y * mul), pack_f16(a.z * mul, a.w * mul), pack_f16(d.x * mul, d.y * mul),
                           pack_f16(d.z * mul, d.w * mul));
        }
    }
}

// The tile's 16 columns of out[T][H], from the experts' outputs y, in slot order.
__device__ __forceinline__ void combine(const FewArgs &g, const int16_t *pei, const uint8_t *slot, int unit, int lane) {
    const int row = lane >> 2;
    if (row >= g.T) return;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const float *y = g.mid + (int64_t)row * g.k * g.H + 16 * unit + 4 * (lane & 3);
#pragma unroll 8
    for (int j = 0; j < g.k; ++j) {
        const int ei = pei[row * g.k + j];
        const float4 v = ei >= 0 ? __ldcg(reinterpret_cast<const float4 *>(y + (int64_t)slot[ei * kMaxTokens + row] * g.H)) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float w = ei >= 0 ? __ldg(g.weights + row * g.k + j) : 0.f;
        o.x += w * v.x;
        o.y += w * v.y;
        o.z += w * v.z;
        o.w += w * v.w;
    }
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
    *reinterpret_cast<uint2 *>(g.out + (int64_t)row * g.H + 16 * unit + 4 * (lane & 3)) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

template <int FMT, bool DOWN, int STAGES>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
k_few(FewArgs g) {
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ uint32_t used[TOPO_GATE_MAX_E / 32];             // experts in use, and how many before each word's
    __shared__ int before[TOPO_GATE_MAX_E / 32];
    __shared__ uint16_t experts[kMaxPairs];
    __shared__ int16_t ids[kMaxPairs], pei[kMaxPairs];          // of each pair: its expert, its place in `experts`
    __shared__ __align__(16) uint8_t slot[kMaxPairs * kMaxTokens];   // a token's lowest slot that names an expert, or 255
    __shared__ uint32_t amax[kMaxRows];                         // of the token rows
    __shared__ int pair_of[kMaxRows];                           // down: the pair of each token row
    __shared__ int16_t seg_row[kMaxRows], seg_n[kMaxRows];      // down: the rows of each expert of a batch
    __shared__ int n_used, batch_end, n_rows, n_done;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = g.warps * 32;
    unsigned char *ring = dyn + warp * STAGES * kStageBytes;
    unsigned char *tok = dyn + g.warps * STAGES * kStageBytes;
    float4 *parts = reinterpret_cast<float4 *>(tok + g.cap_rows * g.bpitch);   // [cap_parts][32]
    const int np = g.T * g.k;
    const int kpad = FMT == TOPO_FMT_EIGHT ? (g.K + 127) & ~127 : (g.K + 255) & ~255;

    // Up: everything before this call is done and seen from here on, and the down kernel,
    // which may start now, can rely on that for the ids and the weights.  The token rows are
    // asked for before the first weights: behind them they came 2 to 3 us later.
    if (!DOWN) {
        pdl_wait();
        pdl_trigger();
    }
    int id = tid < np ? __ldg(g.ids + tid) : -1;
    if (!DOWN) {
        for (int row = 0; row < g.T; ++row)
            for (int c = tid; c < kpad / 8; c += threads)
                copy_or_zero(smem_at(tok + row * g.bpitch + 16 * c), c < g.K / 8 ? g.x + (int64_t)row * g.K + 8 * c : g.x, c < g.K / 8);
        copies_end();
        if (blockIdx.x == 0)
            for (int i = tid; i < g.H / 16; i += threads) g.count[i] = 0;
    }
    for (int i = tid; i < TOPO_GATE_MAX_E / 32; i += threads) used[i] = 0;
    for (int i = tid; i < np * kMaxTokens / 4; i += threads) reinterpret_cast<uint32_t *>(slot)[i] = 0xffffffffu;
    __syncthreads();
    for (int i = tid; i < np; i += threads) {
        if (i != tid) id = __ldg(g.ids + i);
        const bool ok = (unsigned)id < (unsigned)g.E;
        ids[i] = ok ? (int16_t)id : (int16_t)-1;
        if (ok) atomicOr(&used[id >> 5], 1u << (id & 31));
        else if (!DOWN && blockIdx.x == 0) set_error(g.hdr, TOPO_ERANGE);
    }
    __syncthreads();
    if (warp == 0) {                                            // the experts in use, in ascending order
        uint32_t w = used[lane];
        const int n = __popc(w);
        int at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += u;
        }
        if (lane == 31) n_used = at;
        at -= n;
        before[lane] = at;
        for (; w; w &= w - 1) experts[at++] = (uint16_t)(32 * lane + __ffs(w) - 1);
    }
    __syncthreads();
    for (int i = tid; i < np; i += threads) {
        const int e = ids[i], t = i / g.k, j = i - t * g.k;
        const int ei = e < 0 ? -1 : before[e >> 5] + __popc(used[e >> 5] & ((1u << (e & 31)) - 1));
        pei[i] = (int16_t)ei;
        int f = 0;
        while (ids[t * g.k + f] != e) ++f;
        if (e >= 0 && f == j) slot[ei * kMaxTokens + t] = (uint8_t)j;
    }
    const int total = n_used * g.units;                         // at most 512 * 4096
    if (DOWN && total == 0) {                                   // no expert at all
        pdl_wait();
        for (int i = blockIdx.x * threads + tid; i < g.T * g.H / 2; i += gridDim.x * threads) reinterpret_cast<uint32_t *>(g.out)[i] = 0;
        return;
    }
    const int begin = (int)((int64_t)total * blockIdx.x / gridDim.x), hi = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
    // Batches of items: up: all of them; down: of as many experts as there is room for the
    // activations of their tokens.
    for (int lo = begin; lo < hi;) {
        const int ei0 = lo / g.units;
        int end = hi;
        if (DOWN) {
            __syncthreads();                                    // `slot`; the batch before is through with its rows
            if (warp == 0) {
                int at = lo, rows = 0;
                for (int i = 0; i < kMaxRows && at < hi; ++i) {
                    const unsigned m = __ballot_sync(0xffffffffu, lane < g.T && slot[(ei0 + i) * kMaxTokens + (lane & (kMaxTokens - 1))] != 255);
                    const int n = __popc(m);
                    if (rows + n > g.cap_rows) break;
                    if (m >> lane & 1u) pair_of[rows + __popc(m & ((1u << lane) - 1))] = lane * g.k + slot[(ei0 + i) * kMaxTokens + lane];
                    if (lane == 0) {
                        seg_row[i] = (int16_t)rows;
                        seg_n[i] = (int16_t)n;
                    }
                    rows += n;
                    at = min(hi, (ei0 + i + 1) * g.units);
                }
                if (lane == 0) {
                    batch_end = at;
                    n_rows = rows;
                }
            }
            __syncthreads();
            end = batch_end;
        }
        // A unit's contraction may be split over 2^log_s warps, so that the warps end together
        const int nu = end - lo;
        int log_s = 0;
        for (int s = 1, best = (nu + g.warps - 1) / g.warps * 16; s <= 4; ++s) {
            const int cost = ((nu << s) + g.warps - 1) / g.warps * (16 >> s);
            if (nu << s <= g.cap_parts && 1 << s <= g.nc && cost < best) {
                best = cost;
                log_s = s;
            }
        }
        const int nitem = nu << log_s;
        Feed<FMT, DOWN> feed;
        feed.item = warp;
        int put = 0, get = 0;
        auto open = [&]() {
            const int gi = lo + (feed.item >> log_s), ei = gi / g.units;
            feed.begin(g, experts[ei], gi - ei * g.units, feed.item & ((1 << log_s) - 1), log_s, lane);
        };
        auto next = [&]() {
            if (feed.item < nitem) {
                feed.issue(g, ring + put * kStageBytes, lane);
                if (++feed.chunk == feed.last) {
                    feed.item += g.warps;
                    if (feed.item < nitem) open();
                }
            }
            copies_end();
            if (++put == STAGES) put = 0;
        };
        __syncwarp();                                           // the ring's last stages were read
        if (feed.item < nitem) open();
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) next();

        // token rows: up: all tokens; down: the activations of the batch's pairs
        if (DOWN && lo == begin) {
            pdl_wait();
            pdl_trigger();
        }
        if (tid < kMaxRows) amax[tid] = 0;
        if (!DOWN) copies_wait<STAGES - 1>();                   // the token rows, all but the weights
        __syncthreads();
        {
            const int rows = DOWN ? n_rows : g.T;
            const int wpr = max(1, g.warps / rows);             // warps to a row
            const int dc = 32 * wpr;
            for (int r0 = 0; r0 < rows; r0 += g.warps) {        // once, but for few warps
                const int row = r0 + warp / wpr, c0 = warp % wpr * 32 + lane;
                const bool on = row < rows && warp < wpr * rows;
                if (DOWN) load_act<FMT>(g, tok, amax, on, row, on ? pair_of[row] : 0, c0, dc, kpad);
                else convert_rows(tok + row * g.bpitch, &amax[on ? row : 0], on, c0, dc, kpad);
            }
        }
        __syncthreads();

        // one unit's sums, whole: lane l holds rows l / 4 and l / 4 + 8 of columns 2 (l % 4) and the next
        auto finish = [&](int ei, int unit, const float (&acc)[4], float r0, float r1) {
            const int r = lane >> 2, t = lane & 3;
            const int row0 = DOWN ? seg_row[ei - ei0] : 0, ncol = DOWN ? seg_n[ei - ei0] : g.T;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = 2 * t + h;
                if (c >= ncol) continue;
                const float s = pow2(row_exp(amax[row0 + c]));
                const float v0 = acc[h] * r0 * s, v1 = acc[2 + h] * r1 * s;
                if (DOWN) {
                    float *y = g.mid + (int64_t)pair_of[row0 + c] * g.H + 16 * unit;
                    __stcg(y + r, v0);
                    __stcg(y + r + 8, v1);
                } else {
                    const int j = slot[ei * kMaxTokens + c];
                    if (j != 255) __stcg(g.mid + ((int64_t)c * g.k + j) * g.I + 8 * unit + r, v0 / (1.f + expf(-v0)) * v1);
                }
            }
        };
        auto row_scales = [&](int ei, int unit, float &r0, float &r1) {
            r0 = r1 = 1.f;
            if (FMT == TOPO_FMT_NV) {
                const float *rs = g.row_scale + (int64_t)experts[ei] * g.rows;
                r0 = __ldg(rs + Feed<FMT, DOWN>::row_of(g, unit, lane >> 2));
                r1 = __ldg(rs + Feed<FMT, DOWN>::row_of(g, unit, (lane >> 2) + 8));
            }
        };

        for (int item = warp; item < nitem; item += g.warps) {
            const int gi = lo + (item >> log_s), ei = gi / g.units, unit = gi - ei * g.units, part = item & ((1 << log_s) - 1);
            // this lane's token column; past the last: any row
            const int row = DOWN ? seg_row[ei - ei0] + min(lane >> 2, seg_n[ei - ei0] - 1) : min(lane >> 2, g.T - 1);
            const unsigned char *col = tok + row * g.bpitch;
            float r0, r1, acc[4] = {0.f, 0.f, 0.f, 0.f};
            if (log_s == 0) row_scales(ei, unit, r0, r1);
            const int c1 = ((part + 1) * g.nc) >> log_s;
            for (int c = (part * g.nc) >> log_s; c < c1; ++c) {
                copies_wait<STAGES - 2>();
                __syncwarp();                                   // every lane's copies are in, its reads of the stage before done
                next();
                stage_product<FMT>(acc, ring + get * kStageBytes, col + c * (FMT == TOPO_FMT_EIGHT ? 256 : 512), lane);
                if (++get == STAGES) get = 0;
            }
            if (log_s == 0) finish(ei, unit, acc, r0, r1);
            else parts[item * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        }
        if (log_s > 0) {
            __syncthreads();
            for (int u = warp; u < nu; u += g.warps) {
                const int ei = (lo + u) / g.units, unit = lo + u - ei * g.units;
                float r0, r1;
                row_scales(ei, unit, r0, r1);
                float4 s = parts[(u << log_s) * 32 + lane];
                for (int p = 1; p < 1 << log_s; ++p) {
                    const float4 v = parts[((u << log_s) + p) * 32 + lane];
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
                const float acc[4] = {s.x, s.y, s.z, s.w};
                finish(ei, unit, acc, r0, r1);
            }
        }
        lo = end;
    }
    copies_wait<0>();
    if (!DOWN) return;
    if (begin == hi) pdl_wait();                                // as the kernels that follow rely on it
    // Whoever brings a tile's last expert adds the tile's columns over the slots.  The fence
    // comes once, after all items: it waits for the warp's copies as well.
    int *list = reinterpret_cast<int *>(dyn);
    if (tid == 0) n_done = 0;
    __syncthreads();
    __threadfence();
    for (int i = begin + tid; i < hi; i += threads)
        if (atomicAdd(g.count + i % g.units, 1) == n_used - 1) list[atomicAdd(&n_done, 1)] = i % g.units;
    __syncthreads();
    __threadfence();
    for (int i = warp; i < n_done; i += g.warps) combine(g, pei, slot, list[i], lane);
}

// ------------------------------------------------------------------------ host
constexpr size_t kFewSmem = 218 * 1024;           // dynamic; the tables take 8 KB

int token_pitch(int K, int fmt) {                 // 16 or 64 bytes past a multiple of 128 (the lanes' bank pattern)
    return fmt == TOPO_FMT_EIGHT ? 2 * ((K + 127) & ~127) + 16 : 2 * ((K + 255) & ~255) + 64;
}

template <int FMT, bool DOWN>
cudaError_t run_few(FewArgs g, cudaStream_t st) {
    auto room = [&](int warps, int stages, int rows) {           // for parts
        return (int64_t)kFewSmem - (int64_t)warps * stages * kStageBytes - (int64_t)rows * g.bpitch;
    };
    int stages = 4;
    g.warps = kMaxWarps;
    if (room(g.warps, stages, g.T) < 16 * 512) stages = 3;
    while (g.warps > 8 && room(g.warps, stages, g.T) < 16 * 512) g.warps -= 2;
    g.cap_rows = g.T;
    while (DOWN && g.cap_rows < kMaxRows && room(g.warps, stages, g.cap_rows + 1) >= 16 * 512) ++g.cap_rows;
    if (room(g.warps, stages, g.cap_rows) < 0) return cudaErrorInvalidValue;
    g.cap_parts = (int)std::min<int64_t>(kMaxParts, room(g.warps, stages, g.cap_rows) / 512);
    const size_t smem = (size_t)g.warps * stages * kStageBytes + (size_t)g.cap_rows * g.bpitch + (size_t)g.cap_parts * 512;
    const auto fn = stages == 4 ? k_few<FMT, DOWN, 4> : k_few<FMT, DOWN, 3>;
    const cudaError_t e = ensure_smem((const void *)fn, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(fn, dim3(kSms), dim3(g.warps * 32), smem, st, g);
}

template <int FMT>
cudaError_t run_both(FewArgs up, FewArgs down, cudaStream_t st) {
    const cudaError_t e = run_few<FMT, false>(up, st);
    return e != cudaSuccess ? e : run_few<FMT, true>(down, st);
}

}  // namespace

size_t few_workspace(int T, int k, int H, int I) {
    return sizeof(WsHeader) + kCounters * sizeof(int32_t) + (size_t)std::min(T, kMaxTokens) * k * ((size_t)H + I) * sizeof(float);
}

cudaError_t launch_expert_few(int T, int E, int k, int H, int I, int fmt, const uint16_t *x, const int32_t *ids,
                              const float *weights, const uint8_t *up, const void *up_scale, const float *up_row,
                              const uint8_t *down, const void *down_scale, const float *down_row, uint16_t *out, void *ws,
                              cudaStream_t st) {
    // tokens of a launch: as many as leave room for the rings of 8 warps
    const int wide = token_pitch(std::max(H, I), fmt);
    const int per = std::min(kMaxTokens, (int)((kFewSmem - 8 * (3 * kStageBytes) - 16 * 512) / wide));
    for (int t0 = 0; t0 < T; t0 += per) {
        FewArgs a = {};
        a.T = std::min(per, T - t0);
        a.E = E;
        a.k = k;
        a.H = H;
        a.I = I;
        a.ids = ids + (int64_t)t0 * k;
        a.weights = weights + (int64_t)t0 * k;
        a.hdr = ws_at<WsHeader>(ws, 0);
        a.count = ws_at<int32_t>(ws, sizeof(WsHeader));
        float *act = ws_at<float>(ws, sizeof(WsHeader) + kCounters * sizeof(int32_t));
        FewArgs d = a;
        const int step = fmt == TOPO_FMT_EIGHT ? 128 : 256;      // values of a stage
        a.x = x + (int64_t)t0 * H;
        a.w = up;
        a.scale = static_cast<const uint8_t *>(up_scale);
        a.row_scale = up_row;
        a.mid = act;
        a.K = H;
        a.rows = 2 * I;
        a.units = I / 8;
        d.act = act;
        d.w = down;
        d.scale = static_cast<const uint8_t *>(down_scale);
        d.row_scale = down_row;
        d.mid = act + (int64_t)std::min(T, kMaxTokens) * k * I;
        d.out = out + (int64_t)t0 * H;
        d.K = I;
        d.rows = H;
        d.units = H / 16;
        for (FewArgs *p : {&a, &d}) {
            p->nc = (p->K + step - 1) / step;
            p->pitch = fmt == TOPO_FMT_EIGHT ? 0 : micro_pitch(p->K, fmt);
            p->bpitch = token_pitch(p->K, fmt);
        }
        const cudaError_t e = fmt == TOPO_FMT_EIGHT ? run_both<TOPO_FMT_EIGHT>(a, d, st)
                              : fmt == TOPO_FMT_MX ? run_both<TOPO_FMT_MX>(a, d, st) : run_both<TOPO_FMT_NV>(a, d, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace topo
