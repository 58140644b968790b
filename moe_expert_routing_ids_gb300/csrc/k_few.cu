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
constexpr int kMaxTokens = 16;                    // of one launch
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
    int warps;
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

// acc += the product of a stage: 16 weight rows, 128 or 256 values, 8 NT token columns.
// K within a stage is dealt to the lanes in whole pieces, the same for weights and tokens.
template <int FMT, int NT>
__device__ __forceinline__ void stage_product(float (&acc)[NT][4], const unsigned char *st, const unsigned char *const (&b)[NT], int lane) {
    const int r = lane >> 2, t = lane & 3;
    const unsigned char *sf = st + 16 * kRowBytes;
    if constexpr (FMT == TOPO_FMT_EIGHT) {
        float d[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[n][i] = 0.f;
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
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 x0 = *reinterpret_cast<const uint4 *>(b[n] + 128 * q + 32 * t);
                const uint4 x1 = *reinterpret_cast<const uint4 *>(b[n] + 128 * q + 32 * t + 16);
                mma16(d[n], f[0], x0.x, x0.y);
                mma16(d[n], f[1], x0.z, x0.w);
                mma16(d[n], f[2], x1.x, x1.y);
                mma16(d[n], f[3], x1.z, x1.w);
            }
        }
        const float2 s = *reinterpret_cast<const float2 *>(sf);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            acc[n][0] += d[n][0] * s.x;
            acc[n][1] += d[n][1] * s.x;
            acc[n][2] += d[n][2] * s.y;
            acc[n][3] += d[n][3] * s.y;
        }
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
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 x = *reinterpret_cast<const uint4 *>(b[n] + 64 * q + 16 * t);
                if (FMT == TOPO_FMT_NV) {
                    mma16(acc[n], a0, x.x, x.y);
                    mma16(acc[n], a1, x.z, x.w);
                } else {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16(d, a0, x.x, x.y);
                    mma16(d, a1, x.z, x.w);
                    acc[n][0] += d[0] * m0;
                    acc[n][1] += d[1] * m0;
                    acc[n][2] += d[2] * m1;
                    acc[n][3] += d[3] * m1;
                }
            }
        }
    }
}

// Issues one warp's stages of an expert's items in order, ahead of their use.
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

template <int FMT, bool DOWN, int NT, int STAGES>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
k_few(FewArgs g) {
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ uint32_t used[TOPO_GATE_MAX_E / 32];
    __shared__ uint16_t experts[TOPO_GATE_MAX_E];
    __shared__ int16_t ids[kMaxTokens * kMaxK];
    __shared__ uint32_t amax[8 * NT];
    __shared__ int pair_of[8 * NT];                             // down: the pair of each column
    __shared__ int n_used, n_col;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = g.warps * 32;
    unsigned char *ring = dyn + warp * STAGES * kStageBytes;
    unsigned char *tok = dyn + g.warps * STAGES * kStageBytes;
    float4 *parts = reinterpret_cast<float4 *>(tok + g.T * g.bpitch);   // [warps][NT][32]
    const int np = g.T * g.k;

    // Up: everything before this call is done and seen from here on, and the down kernel,
    // which may start now, can rely on that for the ids and the weights.
    if (!DOWN) {
        pdl_wait();
        pdl_trigger();
    }
    for (int i = tid; i < TOPO_GATE_MAX_E / 32; i += threads) used[i] = 0;
    __syncthreads();
    for (int i = tid; i < np; i += threads) {
        const int e = __ldg(g.ids + i);
        const bool ok = (unsigned)e < (unsigned)g.E;
        ids[i] = ok ? (int16_t)e : (int16_t)-1;
        if (ok) atomicOr(&used[e >> 5], 1u << (e & 31));
        else if (!DOWN && blockIdx.x == 0) set_error(g.hdr, TOPO_ERANGE);
    }
    if (!DOWN && blockIdx.x == 0)
        for (int i = tid; i < g.H / 16; i += threads) g.count[i] = 0;
    __syncthreads();
    if (warp == 0) {                                            // the experts in use, in ascending order
        uint32_t w = used[lane];
        int n = __popc(w), at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += u;
        }
        if (lane == 31) n_used = at;
        at -= n;
        for (; w; w &= w - 1) experts[at++] = (uint16_t)(32 * lane + __ffs(w) - 1);
    }
    __syncthreads();
    const int64_t total = (int64_t)n_used * g.units;
    if (DOWN && total == 0) {                                   // no expert at all
        pdl_wait();
        for (int i = blockIdx.x * threads + tid; i < g.T * g.H / 2; i += gridDim.x * threads) reinterpret_cast<uint32_t *>(g.out)[i] = 0;
        return;
    }
    int64_t lo = total * blockIdx.x / gridDim.x;
    const int64_t hi = total * (blockIdx.x + 1) / gridDim.x;
    bool first = true;
    while (lo < hi) {
        // the items of one expert: units u0 .. u0 + nu - 1
        const int ei = (int)(lo / g.units), e = experts[ei], u0 = (int)(lo - (int64_t)ei * g.units);
        const int nu = (int)min((int64_t)(g.units - u0), hi - lo);
        lo += nu;
        int log_s = 0;                                          // a unit's contraction is split over 2^log_s warps
        while ((nu << (log_s + 1)) <= g.warps && (1 << (log_s + 1)) <= g.nc) ++log_s;
        const int nitem = nu << log_s;
        Feed<FMT, DOWN> feed;
        feed.item = warp;
        int put = 0, get = 0;
        __syncwarp();                                           // the ring's last stages were read
        auto next = [&]() {
            if (feed.item < nitem) {
                feed.issue(g, ring + put * kStageBytes, lane);
                if (++feed.chunk == feed.last) {
                    feed.item += g.warps;
                    if (feed.item < nitem) feed.begin(g, e, u0 + (feed.item >> log_s), feed.item & ((1 << log_s) - 1), log_s, lane);
                }
            }
            copies_end();
            if (++put == STAGES) put = 0;
        };
        if (feed.item < nitem) feed.begin(g, e, u0 + (feed.item >> log_s), feed.item & ((1 << log_s) - 1), log_s, lane);
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) next();

        if (DOWN || first) {
            // token rows: up: all tokens, once; down: the activations of this expert's pairs
            if (DOWN && first) pdl_wait();
            if (!first) __syncthreads();
            if (tid < 8 * NT) amax[tid] = 0;
            if (DOWN && warp == 0) {
                int first_j = -1;                               // the lowest slot of a token that names e
                if (lane < g.T)
                    for (int j = g.k - 1; j >= 0; --j)
                        if (ids[lane * g.k + j] == e) first_j = j;
                const unsigned m = __ballot_sync(0xffffffffu, first_j >= 0);
                if (first_j >= 0) pair_of[__popc(m & ((1u << lane) - 1))] = lane * g.k + first_j;
                if (lane == 0) n_col = __popc(m);
            }
            __syncthreads();
            const int rows = DOWN ? n_col : g.T;
            const int wpr = max(1, g.warps / rows);             // warps to a row
            const int kpad = FMT == TOPO_FMT_EIGHT ? (g.K + 127) & ~127 : (g.K + 255) & ~255;
            for (int pass = 0; pass < 2; ++pass) {
                for (int v = warp; v < rows * wpr; v += g.warps) {
                    const int row = v / wpr;
                    uint32_t m = 0;
                    const float mul = pass ? pow2(-row_exp(amax[row])) : 0.f;
                    for (int c = (v - row * wpr) * 32 + lane; c < (pass ? kpad : g.K) / 8; c += wpr * 32) {
                        float f[8];
                        if (c < g.K / 8) {
                            if (DOWN) {
                                const float4 *p = reinterpret_cast<const float4 *>(g.act + (int64_t)pair_of[row] * g.K) + 2 * c;
                                const float4 a = __ldcg(p), d = __ldcg(p + 1);
                                f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = d.x, f[5] = d.y, f[6] = d.z, f[7] = d.w;
                            } else {
                                const uint4 a = __ldg(reinterpret_cast<const uint4 *>(g.x + (int64_t)row * g.K) + c);
                                const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                                for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[i] = 0.f;
                        }
                        if (pass == 0) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const uint32_t u = __float_as_uint(f[i]) & 0x7fffffffu;
                                if (u < 0x7f800000u) m = max(m, u);
                            }
                        } else {
                            *reinterpret_cast<uint4 *>(tok + row * g.bpitch + 16 * c) =
                                make_uint4(pack_f16(f[0] * mul, f[1] * mul), pack_f16(f[2] * mul, f[3] * mul),
                                           pack_f16(f[4] * mul, f[5] * mul), pack_f16(f[6] * mul, f[7] * mul));
                        }
                    }
                    if (pass == 0) {
                        m = __reduce_max_sync(0xffffffffu, m);
                        if (lane == 0) atomicMax(&amax[row], m);
                    }
                }
                __syncthreads();
            }
        }
        first = false;
        const int ncol = DOWN ? n_col : g.T;
        const unsigned char *col[NT];                           // this lane's token columns; past the last: any row
#pragma unroll
        for (int n = 0; n < NT; ++n) col[n] = tok + min(8 * n + (lane >> 2), ncol - 1) * g.bpitch;

        // one unit's sums, whole: lane l holds rows l / 4 and l / 4 + 8 of columns 2 (l % 4) and the next
        auto finish = [&](int unit, float (&acc)[NT][4]) {
            const int r = lane >> 2, t = lane & 3;
            float r0 = 1.f, r1 = 1.f;
            if (FMT == TOPO_FMT_NV) {
                const float *rs = g.row_scale + (int64_t)e * g.rows;
                r0 = __ldg(rs + Feed<FMT, DOWN>::row_of(g, unit, r));
                r1 = __ldg(rs + Feed<FMT, DOWN>::row_of(g, unit, r + 8));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = 8 * n + 2 * t + h;
                    if (c >= ncol) continue;
                    const float s = pow2(row_exp(amax[c]));
                    const float v0 = acc[n][h] * r0 * s, v1 = acc[n][2 + h] * r1 * s;
                    if (DOWN) {
                        float *y = g.mid + (int64_t)pair_of[c] * g.H + 16 * unit;
                        __stcg(y + r, v0);
                        __stcg(y + r + 8, v1);
                    } else {
                        int j = 0;                              // the lowest slot that names e
                        while (j < g.k && ids[c * g.k + j] != e) ++j;
                        if (j < g.k) g.mid[((int64_t)c * g.k + j) * g.I + 8 * unit + r] = v0 / (1.f + expf(-v0)) * v1;
                    }
                }
            if (DOWN) {
                // the last expert's: add the tile's columns over the slots
                __threadfence();
                __syncwarp();
                int done = 0;
                if (lane == 0) done = atomicAdd(g.count + unit, 1);
                if (__shfl_sync(0xffffffffu, done, 0) != n_used - 1) return;
                __threadfence();
                for (int row = r; row < g.T; row += 8) {
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float *y = g.mid + (int64_t)row * g.k * g.H + 16 * unit + 4 * t;
#pragma unroll 8
                    for (int j = 0; j < g.k; ++j) {
                        const int id = ids[row * g.k + j];
                        if (id < 0) continue;
                        int f = 0;
                        while (ids[row * g.k + f] != id) ++f;
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(y + (int64_t)f * g.H));
                        const float w = __ldg(g.weights + row * g.k + j);
                        o.x += w * v.x;
                        o.y += w * v.y;
                        o.z += w * v.z;
                        o.w += w * v.w;
                    }
                    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
                    *reinterpret_cast<uint2 *>(g.out + (int64_t)row * g.H + 16 * unit + 4 * t) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
                }
            }
        };

        for (int item = warp; item < nitem; item += g.warps) {
            const int unit = u0 + (item >> log_s), part = item & ((1 << log_s) - 1);
            float acc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
            const int c1 = ((part + 1) * g.nc) >> log_s;
            for (int c = (part * g.nc) >> log_s; c < c1; ++c) {
                copies_wait<STAGES - 2>();
                __syncwarp();                                   // every lane's copies are in, its reads of the stage before done
                next();
                const unsigned char *b[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) b[n] = col[n] + c * (FMT == TOPO_FMT_EIGHT ? 256 : 512);
                stage_product<FMT, NT>(acc, ring + get * kStageBytes, b, lane);
                if (++get == STAGES) get = 0;
            }
            if (log_s == 0) {
                finish(unit, acc);
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n) parts[(item * NT + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
            }
        }
        if (log_s > 0) {
            __syncthreads();
            for (int u = warp; u < nu; u += g.warps) {
                float acc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float4 s = parts[((u << log_s) * NT + n) * 32 + lane];
                    for (int p = 1; p < 1 << log_s; ++p) {
                        const float4 v = parts[(((u << log_s) + p) * NT + n) * 32 + lane];
                        s.x += v.x;
                        s.y += v.y;
                        s.z += v.z;
                        s.w += v.w;
                    }
                    acc[n][0] = s.x, acc[n][1] = s.y, acc[n][2] = s.z, acc[n][3] = s.w;
                }
                finish(u0 + u, acc);
            }
            __syncthreads();
        }
    }
    copies_wait<0>();
    // a CTA without items still has to see the up kernel end, as later calls rely on it
    if (DOWN && first) pdl_wait();
}

// ------------------------------------------------------------------------ host
constexpr size_t kFewSmem = 220 * 1024;           // dynamic; the tables take 7 KB

int token_pitch(int K, int fmt) {                 // 16 or 64 bytes past a multiple of 128 (the lanes' bank pattern)
    return fmt == TOPO_FMT_EIGHT ? 2 * ((K + 127) & ~127) + 16 : 2 * ((K + 255) & ~255) + 64;
}

template <int FMT, bool DOWN, int NT>
cudaError_t run_few(FewArgs g, cudaStream_t st) {
    const int fixed = g.T * g.bpitch;
    auto bytes = [&](int warps, int stages) { return (size_t)warps * (stages * kStageBytes + NT * 512) + fixed; };
    int stages = 4;
    g.warps = kMaxWarps;
    if (bytes(g.warps, stages) > kFewSmem) stages = 3;
    while (g.warps > 4 && bytes(g.warps, stages) > kFewSmem) g.warps -= 2;
    const size_t smem = bytes(g.warps, stages);
    if (smem > kFewSmem) return cudaErrorInvalidValue;
    const auto fn = stages == 4 ? k_few<FMT, DOWN, NT, 4> : k_few<FMT, DOWN, NT, 3>;
    const cudaError_t e = ensure_smem((const void *)fn, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(fn, dim3(kSms), dim3(g.warps * 32), smem, st, g);
}

template <int FMT>
cudaError_t run_both(FewArgs up, FewArgs down, cudaStream_t st) {
    const cudaError_t e = run_few<FMT, false, 1>(up, st);
    return e != cudaSuccess ? e : run_few<FMT, true, 1>(down, st);
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
    const int per = std::min(8, (int)((kFewSmem - 8 * (3 * kStageBytes + 512)) / wide));
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
