// The experts' matrix products in e4m3 with one float32 scale for each block
// of 128 values along the contraction.
//
//   product   y[r][n]     = sum_b sa[r][b] * sw[e][n / 128][b] * (sum over k in block b of a[r][k] * w[e][n][k])
//             for the rows r of each segment of the dispatch layout, e the segment's weights
//   gradient  dw[i][n][k] = sum_b sdy[b][n] * sx[b][k] * (sum over t in block b of dy[n][t] * x[k][t])
//             b over the 128-row blocks of segment i, dy and x laid out column by column
//
// A block's inner sum runs on the tensor cores (tcgen05.mma kind::f8f6f4, four
// steps of 32 into float32 tensor memory); scaling it and adding it to the
// tile's float32 sums in registers is one packed multiply-add for two values.
// Persistent CTAs, one per SM: one thread streams operand tiles with TMA
// through a ring of shared-memory stages, one thread issues the products into
// two alternating tensor-memory accumulators of 256 columns, and eight warps
// scale and add the accumulator that is complete, 128 columns of a row to a
// thread, then store the tile.
//
// Three assignments of the operands to the tile's 128 rows (M) and up to 256
// columns (N):
//   kRowsM  rows of the layout on M, weights on N: the scale of a row is one
//           value per thread.  For long segments.
//   kRowsN  weights on M, rows of the layout on N (a multiple of 16, up to
//           nt): a segment of few rows fills no more of the tile than it has.
//   kGrad   the gradient: n on M, k on N, one segment's blocks contracted.
// Segments start at any row: a tile's loads may run past its segment's last
// row into the next one, those rows are computed and not stored.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "tcgen.cuh"

namespace topo {
namespace {

enum { kRowsM = 0, kRowsN = 1, kGrad = 2 };

constexpr int kKB = 128;                          // contraction values of a block: one 128-byte swizzle row
constexpr int kTileM = 128;
constexpr int kTileN = 256;
constexpr int kSumWarps = 8;                      // warps that scale, add and store
constexpr int kThreads = (kSumWarps + 4) * 32;    // two summing warpgroups, one of producer, issuer and two idle warps
constexpr int kSumRegs = 224, kIoRegs = 56;       // 2 * 128 * 224 + 128 * 56 = 384 * 168, the launch's share
constexpr int kTmemCols = 512;                    // two accumulators of 256 columns
constexpr uint32_t kABytes = kTileM * kKB;
constexpr int kMaxStages = 10;
constexpr int kSegCap = 1024;                     // segments of one launch (the table in shared memory)
constexpr size_t kSmemBytes = 200 * 1024;         // operand ring
constexpr int kMaxSm = 152;

struct GemmArgs {
    const int32_t *seg_off;     // [nseg + 1]
    const int32_t *seg_all;     // kGrad: the offsets from segment 0
    const int32_t *seg_w;       // [nseg] weights of each segment, or null: the segment's index + seg0
    const float *a_scale;       // kRowsM, kRowsN: [rows][KB]; kGrad: [cap / 128][N]
    const float *b_scale;       // kRowsM, kRowsN: [n_w][NB][KB]; kGrad: [cap / 128][K]
    void *out;
    WsHeader *hdr;
    int64_t rows;               // rows of the layout
    int64_t cap;                // kGrad: columns of the transposed operands
    int nseg, seg0, n_w;
    int N, K;                   // kGrad: dw is [N][K]
    int KB, NB;                 // 128-blocks of K and N
    int nt;                     // kRowsN: rows of the layout a tile takes (a multiple of 16); else 256
    int stages;
    uint32_t stage_bytes;
    int out_bf16;
};

struct Tile {
    int seg, w;        // segment, its weights
    int m0, n0;        // first row of A and of B (kRowsM: layout row, weight row within the expert; ...)
    int mlim, nlim;    // rows of A and of B that count, from m0 and n0
    int ncols;         // columns computed (a multiple of 16)
    int kb0, nkb;      // blocks contracted
};

template <int MODE>
__device__ __forceinline__ int tiles_of(const GemmArgs &g, int len) {
    if (MODE == kGrad) return ((g.N + kTileM - 1) / kTileM) * ((g.K + kTileN - 1) / kTileN);
    if (MODE == kRowsM) return ((len + kTileM - 1) / kTileM) * ((g.N + kTileN - 1) / kTileN);
    return ((len + g.nt - 1) / g.nt) * ((g.N + kTileM - 1) / kTileM);
}

// Tile t: its segment by binary search over the exclusive prefix tp[0..nseg].
// Within a segment the layout-row tiles of one weight tile are neighbours, so
// that CTAs running together share the weights through L2.
template <int MODE>
__device__ __forceinline__ Tile find_tile(const GemmArgs &g, const int *tp, const int *so, const int *pad, int t) {
    int lo = 0, hi = g.nseg - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tp[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    Tile r;
    r.seg = lo;
    const int loc = t - tp[lo], len = so[lo + 1] - so[lo];
    r.w = 0;
    if (MODE != kGrad) r.w = g.seg_w ? __ldg(g.seg_w + lo) : g.seg0 + lo;
    if (MODE == kRowsM) {
        const int nm = (len + kTileM - 1) / kTileM, m = loc % nm, n = loc / nm;
        r.m0 = so[lo] + m * kTileM;
        r.mlim = min(kTileM, len - m * kTileM);
        r.n0 = n * kTileN;
        r.nlim = min(kTileN, g.N - r.n0);
        r.ncols = (r.nlim + 15) & ~15;
        r.kb0 = 0;
        r.nkb = g.KB;
    } else if (MODE == kRowsN) {
        const int nn = (len + g.nt - 1) / g.nt, n = loc % nn, m = loc / nn;
        r.m0 = m * kTileM;
        r.mlim = min(kTileM, g.N - r.m0);
        r.n0 = so[lo] + n * g.nt;
        r.nlim = min(g.nt, len - n * g.nt);
        r.ncols = (r.nlim + 15) & ~15;
        r.kb0 = 0;
        r.nkb = g.KB;
    } else {
        const int nm = (g.N + kTileM - 1) / kTileM, m = loc % nm, n = loc / nm;
        r.m0 = m * kTileM;
        r.mlim = min(kTileM, g.N - r.m0);
        r.n0 = n * kTileN;
        r.nlim = min(kTileN, g.K - r.n0);
        r.ncols = (r.nlim + 15) & ~15;
        r.kb0 = pad[lo];
        r.nkb = pad[lo + 1] - pad[lo];
    }
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// acc[c] += scale * D[row][c] for the first 32 * NC columns of this half: 32
// columns are read while the 32 before them are added.  Columns past the
// tile's hold whatever the accumulator held; they are never stored.
template <int MODE, int NC>
__device__ __forceinline__ void add_block(float2 (&acc)[64], uint32_t ta, float r, const float *cs) {
    const float2 rr = make_float2(r, r);
    uint32_t v[2][32];
    tc::tmem_ld(ta, v[0]);
    tc::tmem_wait(v[0]);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (c + 1 < NC) tc::tmem_ld(ta + 32 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 p = make_float2(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1]));
            float2 &d = acc[16 * c + i];
            if (MODE == kRowsM) {
                tc::fma2(d, p, rr);
            } else {
                const float2 k2 = *reinterpret_cast<const float2 *>(cs + 32 * c + 2 * i);
                if (MODE == kRowsN) tc::fma2(d, p, k2);
                else tc::fma2(d, tc::mul2(p, k2), rr);
            }
        }
        if (c + 1 < NC) tc::tmem_wait(v[(c + 1) & 1]);
    }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
k_experts(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, GemmArgs g) {
    extern __shared__ __align__(1024) unsigned char ring[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    __shared__ int expired;
    __shared__ int so[kSegCap + 1], tp[kSegCap + 1], pad[MODE == kGrad ? kSegCap + 1 : 1];
    __shared__ __align__(16) float cs[2][2][128];      // [accumulator][half][column]: scales of the columns
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kSumWarps + 1) tc::tmem_alloc(&tmem_slot, kTmemCols);
    if (tid == 0) {
        for (int s = 0; s < g.stages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&acc_full[b], 1);
            tc::mbar_init(&acc_empty[b], kSumWarps);
        }
        tc::mbar_init(&drained, 1);
        tc::mbar_init_fence();
        expired = 0;
    }
    if (tid == kSumWarps * 32) {
        tc::tma_prefetch(&map_a);
        tc::tma_prefetch(&map_b);
    }
    // the segments' row offsets, then the exclusive prefix of their tile counts;
    // a segment outside the layout or without weights has no tiles and is reported
    for (int i = tid; i <= g.nseg; i += kThreads) so[i] = __ldg(g.seg_off + i);
    __syncthreads();
    if (warp == 0) {
        int run = 0, prun = 0;
        const int lim = (int)g.rows, cap = (int)(g.cap / kKB);
        if (MODE == kGrad) {                       // blocks of the segments of earlier launches
            for (int i = lane; i < g.seg0; i += 32) {
                const int a = __ldg(g.seg_all + i), b = __ldg(g.seg_all + i + 1);
                if (a >= 0 && b >= a && b <= lim) prun += (b - a + kKB - 1) / kKB;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) prun += __shfl_xor_sync(0xffffffffu, prun, o);
        }
        for (int i0 = 0; i0 < g.nseg; i0 += 32) {
            const int i = i0 + lane;
            int n = 0, pb = 0;
            if (i < g.nseg) {
                const int a = so[i], b = so[i + 1];
                bool ok = a >= 0 && b >= a && b <= lim;
                if (!ok) set_error(g.hdr, TOPO_ESTATE);
                if (MODE != kGrad) {
                    const int w = g.seg_w ? __ldg(g.seg_w + i) : g.seg0 + i;
                    if (b > a && (unsigned)w >= (unsigned)g.n_w) {
                        set_error(g.hdr, TOPO_ERANGE);
                        ok = false;
                    }
                }
                if (MODE == kGrad && ok) pb = (b - a + kKB - 1) / kKB;
                if (MODE == kGrad || ok) n = tiles_of<MODE>(g, b - a);
            }
            int x = n, y = pb;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) {
                    x += u;
                    y += v;
                }
            }
            if (i < g.nseg) {
                tp[i] = run + x - n;
                if (MODE == kGrad) {
                    if (prun + y > cap) set_error(g.hdr, TOPO_ESTATE);   // more blocks than the operands hold
                    pad[i] = min(prun + y - pb, cap);
                    if (i == g.nseg - 1) pad[g.nseg] = min(prun + y, cap);
                }
            }
            run += __shfl_sync(0xffffffffu, x, 31);
            prun += __shfl_sync(0xffffffffu, y, 31);
        }
        if (lane == 0) tp[g.nseg] = run;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tmem_slot;
    const int ntiles = tp[g.nseg];

    if (warp >= kSumWarps) {
        tc::regs_dec<kIoRegs>();
    if (warp == kSumWarps) {
        // ------------------------------------------------------------- producer
        if (lane == 0) {
            int s = 0, fill = 0;                       // stage, and how often the ring went round
            bool ok = true;
            for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
                const Tile q = find_tile<MODE>(g, tp, so, pad, t);
                const int ya = MODE == kRowsN ? q.w * g.N + q.m0 : q.m0;
                const int yb = MODE == kRowsM ? q.w * g.N + q.n0 : q.n0;
                const uint32_t bbytes = (uint32_t)(MODE == kRowsN ? q.ncols : kTileN) * kKB;
                for (int kb = 0; kb < q.nkb; ++kb) {
                    if (fill > 0 && !tc::mbar_wait(&empty[s], (uint32_t)(fill - 1) & 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = tc::smem_u32(&full[s]);
                    const uint32_t a = tc::smem_u32(ring) + (uint32_t)s * g.stage_bytes, b = a + kABytes;
                    const int x = (q.kb0 + kb) * kKB;
                    tc::mbar_expect_tx(bar, kABytes + bbytes);
                    tc::tma_load(a, &map_a, x, ya, bar);
                    if (MODE == kRowsN)
                        for (int c = 0; c < q.ncols; c += 16) tc::tma_load(b + (uint32_t)c * kKB, &map_b, x, yb + c, bar);
                    else
                        tc::tma_load(b, &map_b, x, yb, bar);
                    if (++s == g.stages) {
                        s = 0;
                        ++fill;
                    }
                }
            }
            if (!ok) atomicExch(&expired, 1);
            // loads in flight land before the CTA ends
            for (int i = 0; i < g.stages; ++i) {
                const int n = fill + (i < s ? 1 : 0);      // fills of stage i
                if (n > 0 && !tc::mbar_wait(&full[i], (uint32_t)(n - 1) & 1u)) atomicExch(&expired, 1);
            }
        }
    } else if (warp == kSumWarps + 1) {
        // --------------------------------------------------------------- issuer
        if (lane == 0) {
            int s = 0, fill = 0, it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
                const Tile q = find_tile<MODE>(g, tp, so, pad, t);
                const uint32_t idesc = tc::idesc_e4m3(kTileM, q.ncols);
                for (int kb = 0; kb < q.nkb; ++kb, ++it) {
                    const int b = it & 1, round = it >> 1;
                    if ((round > 0 && !tc::mbar_wait(&acc_empty[b], (uint32_t)(round - 1) & 1u)) ||
                        !tc::mbar_wait(&full[s], (uint32_t)fill & 1u)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t a = tc::smem_u32(ring) + (uint32_t)s * g.stage_bytes;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        tc::mma_e4m3(tmem + (uint32_t)(b * kTileN), tc::smem_desc(a + 32u * j),
                                     tc::smem_desc(a + kABytes + 32u * j), idesc, j > 0);
                    tc::mma_commit(tc::smem_u32(&empty[s]));
                    tc::mma_commit(tc::smem_u32(&acc_full[b]));
                    if (++s == g.stages) {
                        s = 0;
                        ++fill;
                    }
                }
            }
            tc::mma_commit(tc::smem_u32(&drained));
            if (!tc::mbar_wait(&drained, 0)) ok = false;
            if (!ok) atomicExch(&expired, 1);
        }
    }
    } else {
        tc::regs_inc<kSumRegs>();
        // --------------------------------------------------- scale, add and store
        const int half = warp >> 2;                      // columns 128 * half ..
        const int row = (warp & 3) * 32 + lane;          // row of the tile
        const int c0 = half * 128;
        int it = 0;
        bool ok = true;
        // an expired wait leaves the loops running without waiting, so that the
        // warps of a half keep meeting at their barrier
        for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
            const Tile q = find_tile<MODE>(g, tp, so, pad, t);
            const int ncol = max(0, min(128, q.ncols - c0));     // this half's columns (0, or a multiple of 16)
            float2 acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
            // this thread's scales: of its row (kRowsM, kGrad), and of column c0 + row (kRowsN, kGrad)
            const float *rs = nullptr, *cl = nullptr, *wsc = nullptr;
            if (MODE == kRowsM) {
                rs = row < q.mlim ? g.a_scale + (int64_t)(q.m0 + row) * g.KB : nullptr;
                wsc = g.b_scale + ((int64_t)q.w * g.NB + min(q.n0 / 128 + half, g.NB - 1)) * g.KB;
            } else if (MODE == kRowsN) {
                cl = c0 + row < q.nlim ? g.a_scale + (int64_t)(q.n0 + c0 + row) * g.KB : nullptr;
                wsc = g.b_scale + ((int64_t)q.w * g.NB + q.m0 / 128) * g.KB;
            } else {
                rs = row < q.mlim ? g.a_scale + (int64_t)q.kb0 * g.N + q.m0 + row : nullptr;
                cl = c0 + row < q.nlim ? g.b_scale + (int64_t)q.kb0 * g.K + q.n0 + c0 + row : nullptr;
            }
            // the next block's scales are on their way while this block is summed
            float rn = 0.f, cn = 0.f, wn = 0.f;
            auto fetch = [&](int kb) {
                if (MODE == kRowsM) {
                    rn = rs ? __ldg(rs + kb) : 0.f;
                    wn = __ldg(wsc + kb);
                } else if (MODE == kRowsN) {
                    cn = cl ? __ldg(cl + kb) : 0.f;
                    wn = __ldg(wsc + kb);
                } else {
                    rn = rs ? __ldg(rs + (int64_t)kb * g.N) : 0.f;
                    cn = cl ? __ldg(cl + (int64_t)kb * g.K) : 0.f;
                }
            };
            if (q.nkb > 0) fetch(0);
            for (int kb = 0; kb < q.nkb; ++kb, ++it) {
                const int b = it & 1;
                const float r = MODE == kRowsM ? rn * wn : rn;
                if (MODE != kRowsM) {
                    cs[b][half][row] = MODE == kRowsN ? cn * wn : cn;
                    tc::bar_sync(1 + half, 128);
                }
                if (kb + 1 < q.nkb) fetch(kb + 1);
                if (ok && !tc::mbar_wait(&acc_full[b], (uint32_t)(it >> 1) & 1u)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                tc::fence_after();
                if (ok) {
                    const uint32_t ta = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(b * kTileN + c0);
                    const float *k2 = cs[b][half];
                    if (MODE == kRowsN) {
                        if (ncol > 64) add_block<MODE, 4>(acc, ta, r, k2);
                        else if (ncol > 32) add_block<MODE, 2>(acc, ta, r, k2);
                        else if (ncol > 0) add_block<MODE, 1>(acc, ta, r, k2);
                    } else if (ncol > 0) {
                        add_block<MODE, 4>(acc, ta, r, k2);
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&acc_empty[b]));
            }
            if (!ok) continue;
            if (MODE == kRowsN) {
                // a thread holds one weight row: 32 lanes store 32 neighbours of one layout row
                if (row < q.mlim) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int c = c0 + 2 * i + h;
                            if (c < q.nlim) {
                                const int64_t o = (int64_t)(q.n0 + c) * g.N + q.m0 + row;
                                const float v = h ? acc[i].y : acc[i].x;
                                if (g.out_bf16) static_cast<__nv_bfloat16 *>(g.out)[o] = __float2bfloat16_rn(v);
                                else static_cast<float *>(g.out)[o] = v;
                            }
                        }
                    }
                }
            } else if (row < q.mlim) {
                const int64_t o = MODE == kGrad ? ((int64_t)(g.seg0 + q.seg) * g.N + q.m0 + row) * g.K + q.n0 + c0
                                                : (int64_t)(q.m0 + row) * g.N + q.n0 + c0;
                const int lim = q.nlim - c0;             // columns of this half that count (a multiple of 16)
                if (MODE == kRowsM && g.out_bf16) {
                    uint4 *d = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(g.out) + o);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (8 * i < lim)
                            d[i] = make_uint4(pack_bf16(acc[4 * i].x, acc[4 * i].y), pack_bf16(acc[4 * i + 1].x, acc[4 * i + 1].y),
                                              pack_bf16(acc[4 * i + 2].x, acc[4 * i + 2].y), pack_bf16(acc[4 * i + 3].x, acc[4 * i + 3].y));
                } else {
                    float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(g.out) + o);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (4 * i < lim) d[i] = make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
                }
            }
        }
        if (!ok && lane == 0) atomicExch(&expired, 1);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kSumWarps + 1) tc::tmem_free(tmem, kTmemCols);
    if (tid == 0 && expired) set_error(g.hdr, TOPO_ETIMEOUT);
}

// ------------------------------------------------------------------------ host
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime, so that the library links
// against the runtime only.
EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Map of a row-major byte matrix [rows][cols], read in boxes of box_rows x 128
// bytes in the 128-byte swizzle; bytes past a row's end or the last row read
// as zero.  base and cols are multiples of 16.
cudaError_t make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int box_rows) {
    const EncodeFn f = encode_fn();
    if (!f) return cudaErrorNotSupported;
    const cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)cols};
    const cuuint32_t box[2] = {kKB, (cuuint32_t)box_rows}, es[2] = {1, 1};
    const CUresult r = f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dim, stride, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MODE>
cudaError_t run_experts(GemmArgs g, const CUtensorMap &ma, const CUtensorMap &mb, cudaStream_t st) {
    const int nb = MODE == kRowsN ? g.nt : kTileN;
    g.stage_bytes = kABytes + (uint32_t)nb * kKB;
    g.stages = std::min<int>(kMaxStages, (int)((kSmemBytes - 1024) / g.stage_bytes));
    const size_t smem = (size_t)g.stages * g.stage_bytes;
    cudaError_t e = ensure_smem((const void *)k_experts<MODE>, smem);
    if (e != cudaSuccess) return e;
    k_experts<MODE><<<kMaxSm, kThreads, smem, st>>>(ma, mb, g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_gemm(int nseg, int64_t rows, int n_w, int N, int K, const uint8_t *a, const float *a_scale,
                               const int32_t *seg_off, const int32_t *seg_w, const uint8_t *w, const float *w_scale,
                               void *out, bool bf16, void *ws, cudaStream_t st) {
    GemmArgs g = {};
    g.a_scale = a_scale;
    g.b_scale = w_scale;
    g.out = out;
    g.hdr = ws_at<WsHeader>(ws, 0);
    g.rows = rows;
    g.n_w = n_w;
    g.N = N;
    g.K = K;
    g.KB = (K + kKB - 1) / kKB;
    g.NB = (N + 127) / 128;
    g.out_bf16 = bf16;
    const int64_t avg = rows / nseg;
    const bool rows_m = avg > 192;
    g.nt = avg <= 32 ? 32 : avg <= 64 ? 64 : avg <= 128 ? 128 : 256;
    CUtensorMap mx, mw;
    cudaError_t e;
    if ((e = make_map(&mx, a, rows, K, rows_m ? kTileM : 16)) != cudaSuccess) return e;
    if ((e = make_map(&mw, w, (int64_t)n_w * N, K, rows_m ? kTileN : kTileM)) != cudaSuccess) return e;
    for (int s0 = 0; s0 < nseg; s0 += kSegCap) {
        g.nseg = std::min(kSegCap, nseg - s0);
        g.seg0 = s0;
        g.seg_off = seg_off + s0;
        g.seg_w = seg_w ? seg_w + s0 : nullptr;
        e = rows_m ? run_experts<kRowsM>(g, mx, mw, st) : run_experts<kRowsN>(g, mw, mx, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_expert_wgrad(int nseg, int64_t rows, int N, int K, int64_t cap, const uint8_t *dy, const float *dy_scale,
                                const uint8_t *x, const float *x_scale, const int32_t *seg_off, float *dw, void *ws,
                                cudaStream_t st) {
    GemmArgs g = {};
    g.seg_all = seg_off;
    g.a_scale = dy_scale;
    g.b_scale = x_scale;
    g.out = dw;
    g.hdr = ws_at<WsHeader>(ws, 0);
    g.rows = rows;
    g.cap = cap;
    g.N = N;
    g.K = K;
    g.nt = kTileN;
    CUtensorMap my, mx;
    cudaError_t e;
    if ((e = make_map(&my, dy, N, cap, kTileM)) != cudaSuccess) return e;
    if ((e = make_map(&mx, x, K, cap, kTileN)) != cudaSuccess) return e;
    for (int s0 = 0; s0 < nseg; s0 += kSegCap) {
        g.nseg = std::min(kSegCap, nseg - s0);
        g.seg0 = s0;
        g.seg_off = seg_off + s0;
        if ((e = run_experts<kGrad>(g, my, mx, st)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace topo
