// The experts applied to a few tokens:
//   out[t] = sum_j w[t][j] * W_down[e] (silu(g) * u),  [g | u] = W_up[e] x[t],  e = ids[t][j]
//
// The weights of the experts in use are the traffic; a token's products are next to
// nothing.  Three kernels: up and down, one CTA to an SM, and the sum over the slots.
//
//   groups  the pairs (t, j) sorted by expert, up to 8 pairs of one expert a group: the
//           columns of a product, for which its weights are read once
//   items   a tile of 16 weight rows (8 gate rows and their 8 up rows; 16 rows of W_down)
//           of one group; a CTA takes an equal share of neighbouring items, its warps one
//           after the other, or parts of an item's contraction where that ends sooner
//   weights each warp streams its rows through its own ring of shared memory, 128 bytes of
//           each row a stage, by cp.async: no warp waits for another
//   product mma.sync m16n8k16 in f16 with float32 sums: weight rows on M, pairs on N.
//           e4m3 and e2m1 are f16 values; scales by 128 and by 32 multiply a block's
//           sum, scales by 16 the f16 weights (6 bits: exact)
//   tokens  as f16 over a power of two for each row (its largest magnitude in
//           [2^14, 2^15)): 11 bits, where bf16 has 8.  The up kernel's CTAs hold all tokens'
//           rows or, where they do not fit, those of their items' pairs; the down kernel's
//           hold their items' activations
//   sums    float32 throughout; each pair's outputs go to the workspace and are added in
//           slot order, so no result depends on the order of the CTAs
//
// The down kernel starts as the up kernel's CTAs end (its first weights do not depend on
// it) and waits for all of it before it reads the activations.
//
// Measured (host call after call, E = 256 of 7168 x 2048, k = 8): one token in 8 bits 60 to
// 63 us, 5.6 to 5.9 TB/s of weights, the up kernel's steady part at 7 TB/s; 32 tokens in MX
// 668 to 725 us, 5.3 to 5.7 TB/s.  One token of 2048 x 768 in MX 15 us, in NV 16; 8 tokens of 64
// experts, 4096 x 1408, k = 6, NV 72 to 75 us, 4.5 to 4.7 TB/s.  What bounds it: in 8 bits memory,
// and 3 to 4 us to the first product of either kernel (the ids' round trip, the sort, the
// first items' addresses, the rows' conversion: instructions, not waits); in 4 bits the
// issue of 275 instructions (NV; MX 243) for a stage of 4096 weights at 58 to 63 percent of
// the slots with 16 warps of 128 registers.  Tried: 20 or 24 warps (fewer registers, spills):
// 7 to 50 percent slower; 8 warps, so that both kernels are resident: 9 percent faster for
// the smallest layer, 5 to 25 slower elsewhere; rows of 144 bytes with their scales instead
// of the exclusive or: 5 percent slower; weights first to leave the L2: equal; the last sum
// in the down kernel, by the CTA that brings a tile's last expert: equal at one token,
// much slower at 32 (with it and rings of 16 x 4 the call took 1186 us, without it and with
// rings of 14 x 3 736); the up contraction split over CTAs, so that each holds a part
// of all tokens' rows: 756 us against 709 at 32 tokens, 173 against 125 with 64 experts of
// 4096 x 1408 (items of four stages).  W_down's kernel in MX keeps five words in local memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "rows.cuh"

namespace topo {
namespace {

constexpr int kSms = 152;
constexpr int kMaxWarps = 16;
constexpr int kRowBytes = 128;                    // of a weight row in a stage
constexpr int kSfRow = 16;                        // scale bytes of a row in a stage, at most
constexpr int kStageBytes = 16 * (kRowBytes + kSfRow);
constexpr int kCols = 8;                          // token columns of a product
constexpr int kMaxPairs = 512;                    // of one launch
constexpr int kMaxRows = TOPO_FEW_MAX_TOKENS;     // token rows that a CTA holds
constexpr int kMaxParts = 64;                     // partial tiles that it holds

struct FewArgs {
    const uint16_t *x;          // up: bf16 [T][K]
    const float *act;           // down: the activations [T * k][K]
    const int32_t *ids;         // [T][k]
    const float *weights;       // [T][k]
    const uint8_t *w;           // [E][rows][K]
    const uint8_t *scale;
    const float *row_scale;     // NV
    float *mid;                 // up: act; down: y [T * k][H]
    uint16_t *out;              // [T][H]
    WsHeader *hdr;
    int T, E, k;
    int K, I, H;                // values contracted; the layer's sizes
    int rows;                   // weight rows of an expert
    int units;                  // tiles of 16 rows of an expert
    uint32_t inv_units, inv_warps, inv_k;   // 2^32 over units, warps, k, rounded up (where that is above 1)
    int nc;                     // stages of a row
    int resident;               // up: a CTA holds all tokens' rows; else those of a batch's pairs
    int64_t pitch;              // 4 bits: scale bytes of a row
    int bpitch;                 // bytes of a token row in shared memory
    int cols;                   // pairs of a group, at most kCols
    int warps, cap_rows, cap_parts;
};

__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// n = 16 bytes, or 16 zeros for n = 0
__device__ __forceinline__ void copy_n(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
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

// d = the product.
__device__ __forceinline__ void mma16_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Two e4m3 values as f16.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}
// Two powers of two from their exponents' bytes (255: NaN), as bf16.
__device__ __forceinline__ uint32_t ue8m0x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}
// Eight e2m1 values as f16.
__device__ __forceinline__ void e2m1x8(uint32_t v, uint32_t (&r)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(v));
}
// Two f16 values times one half of s.
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t s, int high) {
    const __half2 f = *reinterpret_cast<const __half2 *>(&s);
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), high ? __high2half2(f) : __low2half2(f));
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
        float d[4];
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
            if (q == 0) mma16_new(d, f[0], x0.x, x0.y);
            else mma16(d, f[0], x0.x, x0.y);
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
        // the scales of rows r and r + 8 for each 32 values (NV: of this lane's half of them), two to a word
        uint32_t s0[4], s1[4];
        if (FMT == TOPO_FMT_NV) {
            const uint4 a = *reinterpret_cast<const uint4 *>(sf + r * 16), c = *reinterpret_cast<const uint4 *>(sf + (r + 8) * 16);
            const uint32_t pick = t < 2 ? 0x6420u : 0x7531u;
            const uint32_t a0 = __byte_perm(a.x, a.y, pick), a1 = __byte_perm(a.z, a.w, pick);
            const uint32_t c0 = __byte_perm(c.x, c.y, pick), c1 = __byte_perm(c.z, c.w, pick);
            s0[0] = e4m3x2(a0), s0[1] = e4m3x2(a0 >> 16), s0[2] = e4m3x2(a1), s0[3] = e4m3x2(a1 >> 16);
            s1[0] = e4m3x2(c0), s1[1] = e4m3x2(c0 >> 16), s1[2] = e4m3x2(c1), s1[3] = e4m3x2(c1 >> 16);
        } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(sf + r * 16), c = *reinterpret_cast<const uint2 *>(sf + (r + 8) * 16);
            s0[0] = ue8m0x2(a.x), s0[1] = ue8m0x2(a.x >> 16), s0[2] = ue8m0x2(a.y), s0[3] = ue8m0x2(a.y >> 16);
            s1[0] = ue8m0x2(c.x), s1[1] = ue8m0x2(c.x >> 16), s1[2] = ue8m0x2(c.y), s1[3] = ue8m0x2(c.y >> 16);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {                           // 32 values, 8 of them this lane's
            uint32_t f0[4], f1[4];
            e2m1x8(*reinterpret_cast<const uint32_t *>(st + r * kRowBytes + piece<FMT>(r, q) + 4 * t), f0);
            e2m1x8(*reinterpret_cast<const uint32_t *>(st + (r + 8) * kRowBytes + piece<FMT>(r, q) + 4 * t), f1);
            if (FMT == TOPO_FMT_NV) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f0[i] = mul2(f0[i], s0[q >> 1], q & 1);
                    f1[i] = mul2(f1[i], s1[q >> 1], q & 1);
                }
            }
            const uint32_t a0[4] = {f0[0], f1[0], f0[1], f1[1]}, a1[4] = {f0[2], f1[2], f0[3], f1[3]};
            const uint4 x = *reinterpret_cast<const uint4 *>(b + 64 * q + 16 * t);
            if (FMT == TOPO_FMT_NV) {
                mma16(acc, a0, x.x, x.y);
                mma16(acc, a1, x.z, x.w);
            } else {
                const float m0 = __uint_as_float(q & 1 ? s0[q >> 1] & 0xffff0000u : s0[q >> 1] << 16);
                const float m1 = __uint_as_float(q & 1 ? s1[q >> 1] & 0xffff0000u : s1[q >> 1] << 16);
                float d[4];
                mma16_new(d, a0, x.x, x.y);
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
    const unsigned char *src[4];                                // this lane's piece of rows lane / 8 + 4 i, in the next stage
    const unsigned char *sf;                                    // this lane's scales there
    int item, left;                                             // the next stage's item, its stages left
    int bytes;                                                  // of the row from this lane's piece on
    uint32_t dst[2];                                            // where the pieces go in a stage, i even and odd

    // First row of a tile in the expert's weights, from row h of the 16.
    static __device__ __forceinline__ int row_of(const FewArgs &g, int unit, int h) {
        return DOWN ? 16 * unit + h : h < 8 ? 8 * unit + h : g.I + 8 * unit + h - 8;
    }
    __device__ __forceinline__ void place(int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) dst[i] = ((lane >> 3) + 4 * i) * kRowBytes + piece<FMT>((lane >> 3) + 4 * i, lane & 7);
    }
    // Stages from .. to of a unit.
    __device__ __forceinline__ void begin(const FewArgs &g, int e, int unit, int from, int to, int lane) {
        left = to - from;
        const int kb = FMT == TOPO_FMT_EIGHT ? g.K : g.K / 2, at = from * kRowBytes + 16 * (lane & 7);
        bytes = kb - at;
#pragma unroll
        for (int i = 0; i < 4; ++i) src[i] = g.w + ((int64_t)e * g.rows + row_of(g, unit, (lane >> 3) + 4 * i)) * kb + at;
        if (FMT == TOPO_FMT_EIGHT) {
            // the float32 of a 128 x 128 block: of the gate rows and of the up rows
            const int nb = (g.rows + 127) / 128, at = e * nb + row_of(g, unit, lane & 1 ? 8 : 0) / 128;
            sf = g.scale + ((int64_t)at * g.nc + from) * 4;
        } else {
            sf = g.scale + ((int64_t)e * g.rows + row_of(g, unit, lane & 15)) * g.pitch + from * (FMT == TOPO_FMT_NV ? 16 : 8);
        }
    }
    __device__ __forceinline__ void issue(uint32_t st, int lane) {
        const int n = bytes > 0 ? 16 : 0;                       // past the row's end: zeros, nothing is read
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            copy_n(st + dst[i & 1] + (i >> 1) * 8 * kRowBytes, src[i], n);
            src[i] += kRowBytes;
        }
        bytes -= kRowBytes;
        const uint32_t ds = st + 16 * kRowBytes;
        if (FMT == TOPO_FMT_EIGHT) {
            if (lane < 2) copy_async<4>(ds + 4 * lane, sf);
        } else if (lane < 16) {
            if (FMT == TOPO_FMT_NV) copy_async<16>(ds + 16 * lane, sf);
            else copy_async<8>(ds + 16 * lane, sf);
        }
        sf += FMT == TOPO_FMT_EIGHT ? 4 : FMT == TOPO_FMT_NV ? 16 : 8;
        --left;
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

__device__ __forceinline__ float gated(float g, float u) { return g / (1.f + expf(-g)) * u; }

// An activation row as f16 in shared memory, in the same pieces; up to kKeep of them stay
// in registers between the row's largest magnitude and the conversion, more are read twice.
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

// The pairs of experts in [0, E) sorted by expert, and the groups of at most `cols` pairs of
// one expert: a group is what the weights' tiles are read for.  Each CTA sorts for itself:
// which pairs a group holds is the same for all of them.
struct Groups {
    uint16_t pair[kMaxPairs];                       // sorted: the pair, its token
    uint8_t token[kMaxPairs];
    uint16_t expert[kMaxPairs];                     // of each group
    uint16_t start[kMaxPairs + 1];                  // its first place
    int warp_sum[8];
    int n;                                          // groups
};

__device__ __forceinline__ int token_of(const FewArgs &g, int pair) { return g.k == 1 ? pair : (int)__umulhi((uint32_t)pair, g.inv_k); }

// np <= 32: each warp does it for itself, all of them writing the same; id: the lane's.
// No barrier: 0.7 us sooner than below at 8 pairs, where the weights' first bytes wait for it.
__device__ __forceinline__ void sort_few_pairs(const FewArgs &g, Groups &s, int np, int id, bool report) {
    const int lane = threadIdx.x & 31;
    const bool in = lane < np, ok = in && (unsigned)id < (unsigned)g.E;
    if (in && !ok && report) set_error(g.hdr, TOPO_ERANGE);
    const int e = ok ? id : g.E;
    int less = 0, same = 0;
    // eight lanes at once: those from np on hold E, which is below none
    for (int q0 = 0; q0 < np; q0 += 8) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int f = __shfl_sync(0xffffffffu, e, q0 + q);
            less += f < e;
            same += f == e && q0 + q < lane;
        }
    }
    const bool opens = ok && same % g.cols == 0;
    const int at = less + same, mine = opens ? at : 64;
    int group = 0;
    for (int q0 = 0; q0 < np; q0 += 8) {
#pragma unroll
        for (int q = 0; q < 8; ++q) group += __shfl_sync(0xffffffffu, mine, q0 + q) < at;
    }
    if (ok) {
        s.pair[at] = (uint16_t)lane;
        s.token[at] = (uint8_t)token_of(g, lane);
        if (opens) {
            s.expert[group] = (uint16_t)e;
            s.start[group] = (uint16_t)at;
        }
    }
    const int n = __popc(__ballot_sync(0xffffffffu, opens)), held = __popc(__ballot_sync(0xffffffffu, ok));
    if (lane == 0) {
        s.n = n;
        s.start[n] = (uint16_t)held;
    }
    __syncwarp();
}

// np <= kMaxPairs; id: this thread's, of pair tid; count: scratch of TOPO_GATE_MAX_E words and
// kMaxPairs half words.  The experts' first places and groups by a sum over shared counters, 4
// to a thread of the first 8 warps.  A pair's place among its expert's by the counter, in any
// order, where one group holds them all, else by the pairs before it.  Ends with a barrier.
__device__ __forceinline__ void sort_pairs(const FewArgs &g, Groups &s, uint32_t *count, int np, int id, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, threads = g.warps * 32;
    int16_t *const key = reinterpret_cast<int16_t *>(count + TOPO_GATE_MAX_E);
    for (int i = tid; i < TOPO_GATE_MAX_E / 4; i += threads) reinterpret_cast<uint4 *>(count)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    int e[kMaxPairs / 256], rank[kMaxPairs / 256];               // 256 threads at least
#pragma unroll
    for (int j = 0; j < kMaxPairs / 256; ++j) {
        const int i = tid + j * threads;
        e[j] = g.E;
        if (i >= np) continue;
        e[j] = j == 0 ? id : __ldg(g.ids + i);
        if ((unsigned)e[j] >= (unsigned)g.E) {
            if (report) set_error(g.hdr, TOPO_ERANGE);
            key[i] = (int16_t)(e[j] = g.E);
        } else {
            key[i] = (int16_t)e[j];
            rank[j] = (int)atomicAdd(count + e[j], 1u);
        }
    }
    __syncthreads();
    uint32_t c[4], sum = 0;                                      // pairs, and groups in the upper half
    if (tid < 256) {
        const uint4 v = reinterpret_cast<const uint4 *>(count)[tid];
        c[0] = v.x, c[1] = v.y, c[2] = v.z, c[3] = v.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] |= (c[i] + g.cols - 1) / g.cols << 16;
            sum += c[i];
        }
    }
    uint32_t at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += u;
    }
    if (tid < 256 && lane == 31) s.warp_sum[tid >> 5] = (int)at;
    __syncthreads();
    at -= sum;
    if (tid < 256) {
        for (int w = 0; w < tid >> 5; ++w) at += (uint32_t)s.warp_sum[w];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int first = (int)(at & 0xffffu), group = (int)(at >> 16);
            count[4 * tid + i] = (uint32_t)first | (c[i] >> 17 ? 1u << 31 : 0u);   // several groups
            for (int k = 0; k < (int)(c[i] >> 16); ++k) {
                s.expert[group + k] = (uint16_t)(4 * tid + i);
                s.start[group + k] = (uint16_t)(first + k * g.cols);
            }
            at += c[i];
        }
        if (tid == 255) {
            s.n = (int)(at >> 16);
            s.start[at >> 16] = (uint16_t)(at & 0xffffu);
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMaxPairs / 256; ++j) {
        const int i = tid + j * threads;
        if (e[j] >= g.E) continue;
        const uint32_t at_e = count[e[j]];
        int to = (int)(at_e & 0xffffu);
        if (at_e >> 31)
            for (int q = 0; q < i; ++q) to += key[q] == e[j];
        else
            to += rank[j];
        s.pair[to] = (uint16_t)i;
        s.token[to] = (uint8_t)token_of(g, i);
    }
    __syncthreads();
}

template <int FMT, bool DOWN, int STAGES>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
k_few(FewArgs g) {
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ Groups grp;
    __shared__ uint32_t amax[kMaxRows];                         // of the token rows
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kStep = FMT == TOPO_FMT_EIGHT ? 128 : 256;    // values of a stage
    unsigned char *ring = dyn + warp * STAGES * kStageBytes;
    const uint32_t ring_at = smem_at(ring);
    unsigned char *tok = dyn + g.warps * STAGES * kStageBytes;
    float4 *parts = reinterpret_cast<float4 *>(tok + g.cap_rows * g.bpitch);   // [cap_parts][32]
    const int np = g.T * g.k;
    const int kpad = g.nc * kStep;
    // token row t to row `to` of the CTA's, as bf16
    auto bring = [&](int t, int to) {
        const uint16_t *src = g.x + (int64_t)t * g.K;
        for (int c = lane; c < kpad / 8; c += 32)
            copy_n(smem_at(tok + to * g.bpitch + 16 * c), 8 * c < g.K ? src + 8 * c : src, 8 * c < g.K ? 16 : 0);
    };

    // Up: everything before this call is done and seen from here on, and the down kernel,
    // which may start now, can rely on that for the ids and the weights.  The token rows are
    // asked for before the first weights: behind them they came 2 to 3 us later.
    if (!DOWN) {
        pdl_wait();
        pdl_trigger();
    }
    const int mine = np <= 32 ? lane : tid;
    const int id = mine < np ? __ldg(g.ids + mine) : -1;
    if (!DOWN && g.resident) {
        for (int row = warp; row < g.T; row += g.warps) bring(row, row);
        copies_end();
    }
    if (np <= 32) sort_few_pairs(g, grp, np, id, !DOWN && blockIdx.x == 0);
    else sort_pairs(g, grp, reinterpret_cast<uint32_t *>(dyn), np, id, !DOWN && blockIdx.x == 0);   // the rings are empty yet
    const int ng = grp.n, total = ng * g.units;                 // at most 512 * 4096
    // Items: units of groups, group by group.  (Unit by unit, where a CTA has room for all
    // pairs' activations, fewer CTAs meet in a unit's sums, but each loads all activations:
    // 2.6 us more for one token's 8 x 2048, against 1 us less at the end.)
    const int begin = (int)((int64_t)total * blockIdx.x / gridDim.x), hi = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
    auto place = [&](int gi, int &group, int &unit) {
        // gi / units, one too many at most (gi < 2^21, units <= 2^12).  Every warp works the
        // items out for itself: with the compiler's divisions that took 1 us
        group = g.units == 1 ? gi : (int)__umulhi((uint32_t)gi, g.inv_units);
        unit = gi - group * g.units;
        if (unit < 0) {
            --group;
            unit += g.units;
        }
    };
    // Batches of items: of as many groups as there is room for the rows of their pairs; all of
    // them where the CTA holds all tokens' rows.
    const bool by_pair = DOWN || !g.resident;
    for (int lo = begin; lo < hi;) {
        int end = hi, row0 = 0, rows = g.T;
        if (by_pair) {
            int g1, unit0;
            place(lo, g1, unit0);
            row0 = grp.start[g1++];
            while (g1 * g.units < hi && grp.start[g1 + 1] - row0 <= g.cap_rows) ++g1;
            end = min(hi, g1 * g.units);
            rows = grp.start[g1] - row0;
            if (lo != begin) __syncthreads();                   // the batch before is through with its rows
            if (!DOWN) {
                for (int row = warp; row < rows; row += g.warps) bring(grp.token[row0 + row], row);
                copies_end();
            }
        }
        // Whole units as long as there is one for each warp; the rest in parts of their
        // contraction, 2^log_s each, so that the warps end together
        const int nu = end - lo, whole = (int)__umulhi((uint32_t)nu, g.inv_warps) * g.warps, rest = nu - whole;
        int log_s = 0;
#pragma unroll
        for (int s = 1, best = rest > 0 ? 16 : 0; s <= 4; ++s) {
            const int cost = (int)__umulhi((uint32_t)((rest << s) + g.warps - 1), g.inv_warps) * (16 >> s);
            if (rest << s <= g.cap_parts && 1 << s <= g.nc && cost < best) {
                best = cost;
                log_s = s;
            }
        }
        const int nitem = whole + (rest << log_s);
        // item -> its unit, and the part's first and last stage
        auto item_of = [&](int item, int &group, int &unit, int &from, int &to) {
            const int r = item - whole;
            place(lo + (r < 0 ? item : whole + (r >> log_s)), group, unit);
            const int part = r & ((1 << log_s) - 1);
            from = r < 0 ? 0 : part * g.nc >> log_s;
            to = r < 0 ? g.nc : (part + 1) * g.nc >> log_s;
        };
        Feed<FMT, DOWN> feed;
        feed.item = warp;
        feed.place(lane);
        int put = 0, get = 0;
        auto open = [&]() {
            int group, unit, from, to;
            item_of(feed.item, group, unit, from, to);
            feed.begin(g, grp.expert[group], unit, from, to, lane);
        };
        auto next = [&]() {
            if (feed.item < nitem) {
                feed.issue(ring_at + put * kStageBytes, lane);
                if (feed.left == 0) {
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

        // token rows: up: as they came, made f16; down: the activations of the batch's pairs
        if (DOWN && lo == begin) {
            pdl_wait();
            pdl_trigger();
        }
        if (tid < kMaxRows) amax[tid] = 0;
        if (!DOWN) copies_wait<STAGES - 1>();                   // the token rows, all but the weights
        __syncthreads();
        {
            const int wpr = max(1, g.warps / rows);             // warps to a row
            const int dc = 32 * wpr;
            for (int r0 = 0; r0 < rows; r0 += g.warps) {        // once, but for few warps
                const int row = r0 + warp / wpr, c0 = warp % wpr * 32 + lane;
                const bool on = row < rows && warp < wpr * rows;
                if (DOWN) load_act(g, tok, amax, on, row, on ? grp.pair[row0 + row] : 0, c0, dc, kpad);
                else convert_rows(tok + row * g.bpitch, &amax[on ? row : 0], on, c0, dc, kpad);
            }
        }
        __syncthreads();

        // one unit's sums, whole: lane l holds rows l / 4 and l / 4 + 8 of columns 2 (l % 4) and the next
        auto finish = [&](int group, int unit, const float (&acc)[4], float r0, float r1) {
            const int r = lane >> 2, at = grp.start[group] + 2 * (lane & 3);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (at + h >= grp.start[group + 1]) continue;
                const int pair = grp.pair[at + h];
                const float s = pow2(row_exp(amax[by_pair ? at + h - row0 : grp.token[at + h]]));
                const float v0 = two_scales(acc[h], r0, s), v1 = two_scales(acc[2 + h], r1, s);
                if (DOWN) {
                    float *y = g.mid + (int64_t)pair * g.H + 16 * unit;
                    __stcg(y + r, v0);
                    __stcg(y + r + 8, v1);
                } else {
                    __stcg(g.mid + (int64_t)pair * g.I + 8 * unit + r, gated(v0, v1));
                }
            }
        };
        auto row_scales = [&](int group, int unit, float &r0, float &r1) {
            r0 = r1 = 1.f;
            if (FMT == TOPO_FMT_NV) {
                const float *rs = g.row_scale + (int64_t)grp.expert[group] * g.rows;
                r0 = __ldg(rs + Feed<FMT, DOWN>::row_of(g, unit, lane >> 2));
                r1 = __ldg(rs + Feed<FMT, DOWN>::row_of(g, unit, (lane >> 2) + 8));
            }
        };

        for (int item = warp; item < nitem; item += g.warps) {
            int group, unit, from, to;
            item_of(item, group, unit, from, to);
            const bool one = item < whole || log_s == 0;
            // this lane's token column; past the last: any row
            const int at = min(grp.start[group] + (lane >> 2), grp.start[group + 1] - 1);
            const unsigned char *col = tok + (by_pair ? at - row0 : grp.token[at]) * g.bpitch;
            float r0, r1, acc[4] = {0.f, 0.f, 0.f, 0.f};
            if (one) row_scales(group, unit, r0, r1);
            for (int c = from; c < to; ++c) {
                copies_wait<STAGES - 2>();
                __syncwarp();                                   // every lane's copies are in, its reads of the stage before done
                next();
                stage_product<FMT>(acc, ring + get * kStageBytes, col + c * 2 * kStep, lane);
                if (++get == STAGES) get = 0;
            }
            if (one) finish(group, unit, acc, r0, r1);
            else parts[(item - whole) * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        }
        if (log_s > 0) {
            __syncthreads();
            for (int u = warp; u < rest; u += g.warps) {
                int group, unit;
                place(lo + whole + u, group, unit);
                float r0, r1;
                row_scales(group, unit, r0, r1);
                float4 s = parts[(u << log_s) * 32 + lane];
                for (int p = 1; p < 1 << log_s; ++p) {
                    const float4 v = parts[((u << log_s) + p) * 32 + lane];
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
                const float acc[4] = {s.x, s.y, s.z, s.w};
                finish(group, unit, acc, r0, r1);
            }
        }
        lo = end;
    }
    copies_wait<0>();
    if (DOWN && begin == hi) pdl_wait();                        // as the kernels that follow rely on it
}

// out[t] = the sum of the pairs' outputs y over the slots, four columns to a thread, eight
// slots' loads on their way at once.  (Done by the CTA that brings a tile's last expert,
// counted with atomics, it took as long at one token and far longer at 32, where that is
// one and the same CTA for nearly all tiles.)
__global__ void __launch_bounds__(128)
k_few_sum(FewArgs g) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x, n4 = g.H / 4;
    const int t = min(i / n4, g.T - 1), q = i - t * n4;
    // the ids and weights are older than the up kernel, for which the down kernel waited
    // before it let this one start
    int id[8];
    float w[8];
    auto slots = [&](int j0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            id[j] = j0 + j < g.k ? __ldg(g.ids + t * g.k + j0 + j) : -1;
            w[j] = j0 + j < g.k ? __ldg(g.weights + t * g.k + j0 + j) : 0.f;
        }
    };
    slots(0);
    pdl_trigger();
    pdl_wait();
    if (i >= g.T * n4) return;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const float *y = g.mid + (int64_t)t * g.k * g.H + 4 * q;
    for (int j0 = 0; j0 < g.k; j0 += 8) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < g.k) v[j] = __ldcg(reinterpret_cast<const float4 *>(y + (int64_t)(j0 + j) * g.H));
        if (j0 > 0) slots(j0);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if ((unsigned)id[j] < (unsigned)g.E) {               // an id outside has no output
                o.x += w[j] * v[j].x;
                o.y += w[j] * v[j].y;
                o.z += w[j] * v[j].z;
                o.w += w[j] * v[j].w;
            }
    }
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
    *reinterpret_cast<uint2 *>(g.out + (int64_t)t * g.H + 4 * q) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// ------------------------------------------------------------------------ host
constexpr size_t kFewSmem = 218 * 1024;           // dynamic; the tables take 4 KB
constexpr int kLeastParts = 16 * 512;

uint32_t over(int n) { return (uint32_t)((((uint64_t)1 << 32) + n - 1) / n); }     // 2^32 / n, for n > 1

// A token row's bytes: 16 or 64 past a multiple of 128 (the lanes' bank pattern).
int token_pitch(int values, int fmt) { return 2 * values + (fmt == TOPO_FMT_EIGHT ? 16 : 64); }

template <int FMT, bool DOWN>
cudaError_t run_few(FewArgs g, cudaStream_t st) {
    auto room = [&](int warps, int stages, int rows) {           // for parts
        return (int64_t)kFewSmem - (int64_t)warps * stages * kStageBytes - (int64_t)rows * g.bpitch;
    };
    int stages = 4;
    g.warps = kMaxWarps;
    g.cols = kCols;
    // all tokens' rows, where they leave 14 warps rings of 3 stages.  Against a batch's rows
    // beside rings of 16 x 4, in 8 bits, MX and NV: 6 tokens of 256 experts, 7168 x 2048, k = 8
    // 317, 217 and 201 us for 321, 212 and 202; 12 of 64, 4096 x 1408, k = 6 133, 91 and 89 for 133, 89
    // and 89; 28 of 64, 2048 x 1024, k = 8 78, 51 and 56 for 75, 50 and 54: next to equal
    g.resident = !DOWN && room(14, 3, g.T) >= kLeastParts;
    if (!g.resident)                                             // rows of a very wide layer
        while (g.cols > 1 && room(8, 3, g.cols) < kLeastParts) --g.cols;
    const int least = g.resident ? g.T : g.cols;
    if (room(g.warps, stages, least) < kLeastParts) stages = 3;
    while (g.warps > 8 && room(g.warps, stages, least) < kLeastParts) g.warps -= 2;
    g.cap_rows = least;
    while (!g.resident && g.cap_rows < kMaxRows && room(g.warps, stages, g.cap_rows + 1) >= kLeastParts) ++g.cap_rows;
    if (room(g.warps, stages, g.cap_rows) < 0) return cudaErrorInvalidValue;
    g.inv_warps = over(g.warps);
    g.cap_parts = (int)std::min<int64_t>(kMaxParts, room(g.warps, stages, g.cap_rows) / 512);
    const size_t smem = (size_t)g.warps * stages * kStageBytes + (size_t)g.cap_rows * g.bpitch + (size_t)g.cap_parts * 512;
    const auto fn = stages == 4 ? k_few<FMT, DOWN, 4> : k_few<FMT, DOWN, 3>;
    const cudaError_t e = ensure_smem((const void *)fn, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(fn, dim3(kSms), dim3(g.warps * 32), smem, st, g);
}

template <int FMT>
cudaError_t run_both(FewArgs up, FewArgs down, cudaStream_t st) {
    cudaError_t e;
    if ((e = run_few<FMT, false>(up, st)) != cudaSuccess) return e;
    if ((e = run_few<FMT, true>(down, st)) != cudaSuccess) return e;
    return launch_pdl(k_few_sum, dim3((unsigned)((down.T * (down.H / 4) + 127) / 128)), dim3(128), 0, st, down);
}

}  // namespace

static int few_tokens(int T, int k) { return std::min(T, kMaxPairs / k); }      // of a launch

size_t few_workspace(int T, int k, int H, int I) {
    return sizeof(WsHeader) + (size_t)few_tokens(T, k) * k * ((size_t)H + I) * sizeof(float);
}

cudaError_t launch_expert_few(int T, int E, int k, int H, int I, int fmt, const uint16_t *x, const int32_t *ids,
                              const float *weights, const uint8_t *up, const void *up_scale, const float *up_row,
                              const uint8_t *down, const void *down_scale, const float *down_row, uint16_t *out, void *ws,
                              cudaStream_t st) {
    const int per = few_tokens(T, k);
    const int step = fmt == TOPO_FMT_EIGHT ? 128 : 256;          // values of a stage
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
        float *y = ws_at<float>(ws, sizeof(WsHeader));
        float *act = y + (int64_t)per * k * H;
        FewArgs d = a;
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
        d.mid = y;
        d.out = out + (int64_t)t0 * H;
        d.K = I;
        d.rows = H;
        d.units = H / 16;
        for (FewArgs *p : {&a, &d}) {
            p->nc = (p->K + step - 1) / step;
            p->inv_units = over(p->units);
            p->inv_k = over(k);
            p->pitch = fmt == TOPO_FMT_EIGHT ? 0 : micro_pitch(p->K, fmt);
        }
        a.bpitch = token_pitch(a.nc * step, fmt);
        d.bpitch = token_pitch(d.nc * step, fmt);
        const cudaError_t e = fmt == TOPO_FMT_EIGHT ? run_both<TOPO_FMT_EIGHT>(a, d, st)
                              : fmt == TOPO_FMT_MX ? run_both<TOPO_FMT_MX>(a, d, st) : run_both<TOPO_FMT_NV>(a, d, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace topo
