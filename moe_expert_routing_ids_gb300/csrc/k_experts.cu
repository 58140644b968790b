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
// tile's float32 sums in registers is one packed multiply-add for two values
// (two for the gradient, whose rows and columns both have scales).
//
// The tile's rows (M, 128 for each CTA) are weight rows n; its columns (N, up
// to 256) are layout rows, or the gradient's k.  A tile takes as many layout
// rows as its segment has, rounded up to 16 (32 for a CTA pair), so ragged
// segments waste no more than that.  Segments start at any row: a tile's loads
// may run past its segment's last row into the next one; those columns are
// computed and not stored.
//
// Persistent CTAs, one per SM: one thread streams operand tiles with TMA
// through a ring of shared-memory stages, one thread issues the products into
// two alternating accumulators of 256 tensor-memory columns, and two
// warpgroups scale and add the one that is complete, 32 rows x 128 columns to
// a warp.  Two warps bring the scales of four blocks at a time to shared memory
// ahead of them (a layout row's scales are consecutive, so a block's are one
// line each: loaded by the summing warps a block ahead, they held them up for
// the whole latency). With CG = 2 two neighbouring SMs work on one tile of 256 rows: each
// holds its own 128 rows and half of the columns' operand, the tensor cores
// read the other half from the neighbour, and a block of 128 x 256 costs a
// CTA 32 KB of shared-memory traffic each way instead of 48 KB.  (One CTA
// alone is held by that traffic: without any summing, 2.7 PFLOP/s.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "tcgen.cuh"

namespace topo {
namespace {

enum { kProduct = 0, kGrad = 1 };

constexpr int kKB = 128;                          // contraction values of a block: one 128-byte swizzle row
constexpr int kTileM = 128;                       // rows of a CTA
constexpr int kTileN = 256;
constexpr int kSumWarps = 8;                      // warps that scale, add and store
constexpr int kThreads = (kSumWarps + 4) * 32;    // two summing warpgroups, one of producer, issuer and two scale warps
// registers of a thread of the summing and of the other warpgroup; 2 * 128 times
// the one and 128 times the other are the launch's 384 * 168
template <int MODE>
constexpr int kSumRegs = MODE == kProduct ? 224 : 216;
template <int MODE>
constexpr int kIoRegs = (384 * 168 - 256 * kSumRegs<MODE>) / 128;
constexpr int kTmemCols = 512;                    // two accumulators of 256 columns
constexpr uint32_t kABytes = kTileM * kKB;
constexpr int kMaxStages = 9;
constexpr int kScaleKB = 4;                       // blocks whose scales are brought together
constexpr int kSegCap = 1024;                     // segments of one launch (the table in shared memory)
constexpr uint32_t kRingBytes = 192 * 1024;       // operand stages
constexpr uint32_t kStageOut = 2048;              // bytes a warp stores through shared memory at a time
constexpr int kSms = 152;

struct GemmArgs {
    const int32_t *seg_off;     // [nseg + 1]
    const int32_t *seg_all;     // gradient: the offsets from segment 0
    const int32_t *seg_w;       // [nseg] weights of each segment, or null: the segment's index + seg0
    const float *w_scale;       // product: [n_w][NB][KB] weights; gradient: [cap / 128][N] of dy
    const float *x_scale;       // product: [rows][KB] layout rows; gradient: [cap / 128][K] of x
    void *out;
    WsHeader *hdr;
    int64_t rows;               // rows of the layout
    int64_t cap;                // gradient: columns of the transposed operands
    int nseg, seg0, n_w;
    int N, K;                   // gradient: dw is [N][K]
    int KB, NB;                 // 128-blocks of K and N
    int nt;                     // columns of a tile: up to 256
    int box;                    // rows of one load of the columns' operand
    int stages;
    uint32_t stage_bytes;
    int out_bf16;
    int vec_scale;              // product: a row's scales can be read four at a time
};

struct Tile {
    int seg, w;        // segment, its weights
    int m0, n0;        // first row and column
    int mlim, nlim;    // rows and columns that count, from m0 and n0
    int ncols;         // columns computed
    int kb0, nkb;      // blocks contracted
};

template <int MODE, int CG>
__device__ __forceinline__ int tiles_of(const GemmArgs &g, int len) {
    const int m = MODE == kProduct ? len : g.N, n = MODE == kProduct ? g.N : g.K;
    return ((m + CG * kTileM - 1) / (CG * kTileM)) * ((n + g.nt - 1) / g.nt);
}

// Tile t: its segment by binary search over the exclusive prefix tp[0..nseg].
// Within a segment the layout-row tiles of one weight tile are neighbours, so
// that CTAs running together share the weights through L2.
template <int MODE, int CG>
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
    const int me = MODE == kProduct ? len : g.N, ne = MODE == kProduct ? g.N : g.K;
    const int nm = (me + CG * kTileM - 1) / (CG * kTileM), n = loc / nm, m = loc - n * nm;
    r.w = MODE == kGrad ? 0 : g.seg_w ? __ldg(g.seg_w + lo) : g.seg0 + lo;
    r.m0 = m * CG * kTileM;
    r.mlim = min(CG * kTileM, me - r.m0);
    r.n0 = n * g.nt;
    r.nlim = min(g.nt, ne - r.n0);
    if (MODE == kProduct) r.m0 += so[lo];
    r.ncols = (r.nlim + 16 * CG - 1) & ~(16 * CG - 1);
    r.kb0 = MODE == kGrad ? pad[lo] : 0;
    r.nkb = MODE == kGrad ? pad[lo + 1] - pad[lo] : g.KB;
    return r;
}

// Place of column c's scale: a lane's columns 8 j + 2 (lane % 4) + 0 .. 1 of two
// neighbouring groups j are 16 consecutive bytes.
__device__ __forceinline__ int scale_at(int c) { return (c & ~15) + ((c >> 1) & 3) * 4 + ((c >> 3) & 1) * 2 + (c & 1); }

__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Sums of a thread.  kProduct: acc[i] holds columns 2 i and 2 i + 1 of row `lane`.
// kGrad: acc[(h * 16 + j) * 2 + r] holds columns 8 j + 2 (lane % 4) and the
// next of row 16 h + 8 r + lane / 4.
using Acc = float2[64];

// kProduct: acc += s * block, 128 columns of this thread's row.  32 columns are
// read while the 32 before them are added.
__device__ __forceinline__ void add_rows(Acc &acc, uint32_t ta, float s) {
    const float2 s2 = make_float2(s, s);
    uint32_t v[2][32];
    tc::tmem_ld_rows(ta, v[0]);
    tc::tmem_wait(v[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (c < 3) tc::tmem_ld_rows(ta + 32 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            tc::fma2(acc[16 * c + i], make_float2(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1])), s2);
        if (c < 3) tc::tmem_wait(v[(c + 1) & 1]);
    }
}

// kGrad: acc += scales * block for NJ groups of 8 columns from group J0.  cs: the
// columns' scales in the order a lane takes them, 4 (two groups) per 16 bytes;
// rs: the rows' scales.
template <int J0, int NJ>
__device__ __forceinline__ void add_cols(Acc &acc, int h, const uint32_t (&v)[4 * NJ], const float *cs, const float (&rs)[4]) {
#pragma unroll
    for (int jj = 0; jj < NJ; jj += 2) {
        const float4 k4 = *reinterpret_cast<const float4 *>(cs + 8 * (J0 + jj));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float2 k2 = u ? make_float2(k4.z, k4.w) : make_float2(k4.x, k4.y);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = 4 * (jj + u) + 2 * r;
                const float2 p = make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                tc::fma2(acc[(h * 16 + J0 + jj + u) * 2 + r], tc::mul2(p, k2), make_float2(rs[2 * h + r], rs[2 * h + r]));
            }
        }
    }
}

// kGrad: 128 columns, 16 rows x 64 columns read while the ones before are added.
__device__ __forceinline__ void add_block(Acc &acc, uint32_t ta, const float *cs, const float (&rs)[4]) {
    constexpr uint32_t kRow16 = 16u << 16;
    uint32_t a[32], b[32];
    tc::tmem_ld(ta, a);
    tc::tmem_wait(a);
    tc::tmem_ld(ta + kRow16, b);
    add_cols<0, 8>(acc, 0, a, cs, rs);
    tc::tmem_wait(b);
    tc::tmem_ld(ta + 64, a);
    add_cols<0, 8>(acc, 1, b, cs, rs);
    tc::tmem_wait(a);
    tc::tmem_ld(ta + 64 + kRow16, b);
    add_cols<8, 8>(acc, 0, a, cs, rs);
    tc::tmem_wait(b);
    add_cols<8, 8>(acc, 1, b, cs, rs);
}

template <int MODE, int CG>
__global__ void __launch_bounds__(kThreads, 1)
k_experts(const __grid_constant__ CUtensorMap map_m, const __grid_constant__ CUtensorMap map_n, GemmArgs g) {
    extern __shared__ __align__(1024) unsigned char ring[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], sc_full[2], sc_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    __shared__ int expired;
    __shared__ int so[kSegCap + 1], tp[kSegCap + 1], pad[MODE == kGrad ? kSegCap + 1 : 1];
    __shared__ __align__(16) float cs[2][kScaleKB][kTileN];    // scales of the columns, see scale_at; kProduct: of the
                                                               // rows, times each half's weight scale
    __shared__ float rsc[MODE == kGrad ? 2 : 1][kScaleKB][kTileM];      // gradient: scales of the rows
    __shared__ __align__(128) unsigned char outs[MODE == kGrad ? 16 : kSumWarps * kStageOut];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? tc::cluster_rank() : 0;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;

    if (warp == kSumWarps + 1) tc::tmem_alloc<CG>(&tmem_slot, kTmemCols);
    if (tid == 0) {
        for (int s = 0; s < g.stages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&acc_full[b], 1);
            tc::mbar_init(&acc_empty[b], CG * kSumWarps);
            tc::mbar_init(&sc_full[b], 2);
            tc::mbar_init(&sc_empty[b], kSumWarps);
        }
        tc::mbar_init(&drained, 1);
        tc::mbar_init_fence();
        expired = 0;
    }
    if (tid == kSumWarps * 32) {
        tc::tma_prefetch(&map_m);
        tc::tma_prefetch(&map_n);
    }
    // the segments' row offsets, then the exclusive prefix of their tile counts;
    // a segment outside the layout or without weights has no tiles and is reported
    for (int i = tid; i <= g.nseg; i += kThreads) so[i] = __ldg(g.seg_off + i);
    __syncthreads();
    if (warp == 0) {
        int run = 0, prun = 0;
        const int lim = (int)g.rows, cap = (int)(g.cap / kKB);
        if (MODE == kGrad) {                                // blocks of the segments of earlier launches
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
                if (MODE == kGrad || ok) n = tiles_of<MODE, CG>(g, b - a);
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
    if (CG == 2) tc::cluster_sync();               // the neighbour's barriers are initialised
    tc::fence_after();

    if (warp >= kSumWarps) {
        tc::regs_dec<kIoRegs<MODE>>();
        const uint32_t tmem = tmem_slot;
        const int ntiles = tp[g.nseg];
        if (warp == kSumWarps) {
            // --------------------------------------------------------- producer
            // CG = 2: both CTAs' loads report to the even CTA's barrier
            int s = 0, fill = 0;                       // stage, and how often the ring went round
            bool ok = true;
            for (int t = first; t < ntiles && ok; t += step) {
                const Tile q = find_tile<MODE, CG>(g, tp, so, pad, t);
                const int ym = q.m0 + (int)rank * kTileM;
                const int nh = q.ncols / CG;                                // this CTA's columns
                const int yn = (MODE == kProduct ? q.w * g.N : 0) + q.n0 + (int)rank * nh;
                const int boxes = (nh + g.box - 1) / g.box;
                const uint32_t bytes = CG * (kABytes + (uint32_t)(boxes * g.box) * kKB);
                for (int kb = 0; kb < q.nkb; ++kb) {
                    if (fill > 0 && !tc::mbar_wait(&empty[s], (uint32_t)(fill - 1) & 1u)) {
                        ok = false;
                        break;
                    }
                    uint32_t bar = tc::smem_u32(&full[s]);
                    if (CG == 2) bar = tc::in_cta(bar, 0);
                    const uint32_t a = tc::smem_u32(ring) + (uint32_t)s * g.stage_bytes, b = a + kABytes;
                    const int x = (q.kb0 + kb) * kKB;
                    if (tc::elect()) {
                        if (rank == 0) tc::mbar_expect_tx(tc::smem_u32(&full[s]), bytes);
                        tc::tma_load<CG>(a, &map_m, x, ym, bar);
                        for (int c = 0; c < boxes; ++c)
                            tc::tma_load<CG>(b + (uint32_t)(c * g.box) * kKB, &map_n, x, yn + c * g.box, bar);
                    }
                    __syncwarp();
                    if (++s == g.stages) {
                        s = 0;
                        ++fill;
                    }
                }
            }
            if (!ok) atomicExch(&expired, 1);
            // loads in flight land before the CTA ends: the barriers tell the even
            // CTA for both; after an expired wait the other one allows them 10 ms
            if (rank == 0) {
                for (int i = 0; i < g.stages; ++i) {
                    const int n = fill + (i < s ? 1 : 0);      // fills of stage i
                    if (n > 0 && !tc::mbar_wait(&full[i], (uint32_t)(n - 1) & 1u)) atomicExch(&expired, 1);
                }
            } else if (!ok) {
                const uint64_t t0 = tc::globaltimer_ns();
                while (tc::globaltimer_ns() - t0 < 10000000ull) {
                }
            }
        } else if (warp == kSumWarps + 1 && rank == 0) {
            // ----------------------------------------------------------- issuer
            int s = 0, fill = 0, it = 0;
            bool ok = true;
            for (int t = first; t < ntiles && ok; t += step) {
                const Tile q = find_tile<MODE, CG>(g, tp, so, pad, t);
                const uint32_t idesc = tc::idesc_e4m3(CG * kTileM, q.ncols);
                for (int kb = 0; kb < q.nkb; ++kb, ++it) {
                    const int b = it & 1, round = it >> 1;
                    if ((round > 0 && !tc::mbar_wait(&acc_empty[b], (uint32_t)(round - 1) & 1u)) ||
                        !tc::mbar_wait(&full[s], (uint32_t)fill & 1u)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t a = tc::smem_u32(ring) + (uint32_t)s * g.stage_bytes;
                    if (tc::elect()) {
                        const uint64_t dm = tc::smem_desc(a), dn = tc::smem_desc(a + kABytes);
#pragma unroll
                        for (int j = 0; j < 4; ++j)            // 32 bytes on within the swizzled row
                            tc::mma_e4m3<CG>(tmem + (uint32_t)(b * kTileN), dm + 2 * j, dn + 2 * j, idesc, j > 0);
                        tc::mma_commit<CG>(tc::smem_u32(&empty[s]));
                        tc::mma_commit<CG>(tc::smem_u32(&acc_full[b]));
                    }
                    __syncwarp();
                    if (++s == g.stages) {
                        s = 0;
                        ++fill;
                    }
                }
            }
            if (tc::elect()) tc::mma_commit<CG>(tc::smem_u32(&drained));
            __syncwarp();
            if (!tc::mbar_wait(&drained, 0)) ok = false;
            if (!ok) atomicExch(&expired, 1);
        } else if (warp >= kSumWarps + 2) {
            // ----------------------------------------------------------- scales
            const int sl = tid - (kSumWarps + 2) * 32;           // 0 .. 63
            int gi = 0;
            bool ok = true;
            for (int t = first; t < ntiles && ok; t += step) {
                const Tile q = find_tile<MODE, CG>(g, tp, so, pad, t);
                const int m1 = q.m0 + (int)rank * kTileM;
                for (int kb = 0; kb < q.nkb; kb += kScaleKB, ++gi) {
                    const int slot = gi & 1, nk = min(kScaleKB, q.nkb - kb);
                    constexpr int kCols = MODE == kProduct ? kTileM / 64 : kTileN / 64;
                    float v[kCols][kScaleKB], w[2][kScaleKB], r[2][kScaleKB];
                    if (MODE != kGrad) {
                        // weight scales of the two halves of the columns
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int nb = min(q.n0 / 128 + h, g.NB - 1);
                            const float *wp = g.w_scale + ((int64_t)q.w * g.NB + nb) * g.KB + kb;
#pragma unroll
                            for (int u = 0; u < kScaleKB; ++u) w[h][u] = u < nk ? __ldg(wp + u) : 0.f;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kCols; ++i) {
                        const int col = sl + 64 * i;
#pragma unroll
                        for (int u = 0; u < kScaleKB; ++u) v[i][u] = 0.f;
                        if (MODE == kGrad) {
                            const float *p = g.x_scale + (int64_t)(q.kb0 + kb) * g.K + q.n0 + col;
                            if (col < q.nlim) {
#pragma unroll
                                for (int u = 0; u < kScaleKB; ++u)
                                    if (u < nk) v[i][u] = __ldg(p + (int64_t)u * g.K);
                            }
                        } else {
                            const bool in = (int)rank * kTileM + col < q.mlim;
                            const float *p = g.x_scale + (int64_t)(m1 + col) * g.KB + kb;
                            if (in && g.vec_scale) {
                                const float4 f = __ldg(reinterpret_cast<const float4 *>(p));
                                v[i][0] = f.x;
                                v[i][1] = f.y;
                                v[i][2] = f.z;
                                v[i][3] = f.w;
                            } else if (in) {
#pragma unroll
                                for (int u = 0; u < kScaleKB; ++u)
                                    if (u < nk) v[i][u] = __ldg(p + u);
                            }
                        }
                    }
                    if (MODE == kGrad) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float *p = g.w_scale + (int64_t)(q.kb0 + kb) * g.N + m1 + sl + 64 * i;
#pragma unroll
                            for (int u = 0; u < kScaleKB; ++u)
                                r[i][u] = u < nk && m1 + sl + 64 * i < g.N ? __ldg(p + (int64_t)u * g.N) : 0.f;
                        }
                    }
                    if (gi >= 2) ok = tc::mbar_wait(&sc_empty[slot], (uint32_t)((gi >> 1) - 1) & 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
#pragma unroll
                        for (int u = 0; u < kScaleKB; ++u) {
                            const int col = sl + 64 * i;
                            if (MODE == kProduct) {
                                cs[slot][u][col] = v[i][u] * w[0][u];
                                cs[slot][u][128 + col] = v[i][u] * w[1][u];
                            } else {
                                cs[slot][u][scale_at(col)] = v[i][u];
                            }
                        }
                    if (MODE == kGrad) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int u = 0; u < kScaleKB; ++u) rsc[slot][u][sl + 64 * i] = r[i][u];
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sc_full[slot]));
                }
            }
            if (!ok && lane == 0) atomicExch(&expired, 1);
        }
    } else {
        tc::regs_inc<kSumRegs<MODE>>();
        const uint32_t tmem = tmem_slot;
        const int ntiles = tp[g.nseg];
        // --------------------------------------------------- scale, add and store
        const int half = warp >> 2, wq = warp & 3;       // columns 128 * half .., rows 32 * wq ..
        const int c0 = half * 128;
        const int quad = lane & 3, r8 = lane >> 2;
        const uint32_t lanes = (uint32_t)(wq * 32) << 16;
        uint32_t done = tc::smem_u32(&acc_empty[0]);     // the even CTA's
        if (CG == 2) done = tc::in_cta(done, 0);
        int it = 0, gi = 0;
        // an expired wait lets these warps run on without waiting (and without
        // storing), so that they reach the end with the rest of the CTA
        for (int t = first; t < ntiles; t += step) {
            int nkb, ncol;
            {
                const Tile q = find_tile<MODE, CG>(g, tp, so, pad, t);
                nkb = q.nkb;
                ncol = max(0, min(128, q.ncols - c0));
            }
            Acc acc;
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
            for (int kb = 0; kb < nkb; ++kb, ++it) {
                const int b = it & 1, u = kb & (kScaleKB - 1), slot = gi & 1;
                if (u == 0) tc::mbar_wait_or(&sc_full[slot], (uint32_t)(gi >> 1) & 1u, &expired);
                float rs[4] = {1.f, 1.f, 1.f, 1.f};
                if (MODE == kProduct) rs[0] = cs[slot][u][c0 + wq * 32 + lane];
                if (MODE == kGrad) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) rs[i] = rsc[MODE == kGrad ? slot : 0][u][wq * 32 + 8 * i + r8];
                }
                tc::mbar_wait_or(&acc_full[b], (uint32_t)(it >> 1) & 1u, &expired);
                __syncwarp();
                tc::fence_after();
                const uint32_t ta = tmem + lanes + (uint32_t)(b * kTileN + c0);
                if (ncol > 0) {
                    if (MODE == kProduct) add_rows(acc, ta, rs[0]);
                    else add_block(acc, ta, &cs[slot][u][c0 + 4 * quad], rs);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) tc::mbar_arrive_cluster(done + 8 * b);
                    else tc::mbar_arrive(done + 8 * b);
                    if (u == kScaleKB - 1 || kb + 1 == nkb) tc::mbar_arrive(tc::smem_u32(&sc_empty[slot]));
                }
                gi += u == kScaleKB - 1 || kb + 1 == nkb;
            }
            if (*(volatile int *)&expired) continue;
            // found again rather than kept in registers over the loop
            const Tile q = find_tile<MODE, CG>(g, tp, so, pad, t);
            const int m1 = (int)rank * kTileM + wq * 32;         // this warp's first row, from m0
            if (MODE == kProduct) {
                if (g.out_bf16) {
                    // 32 rows x 32 values at a time, turned through shared memory so that four
                    // lanes store 64 neighbouring bytes: 16-byte pieces, piece index XOR (row / 2)
                    unsigned char *w = outs + warp * kStageOut;
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(g.out) + (int64_t)(q.m0 + m1 + r8) * g.N + q.n0 + c0 + 8 * quad;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c0 + 32 * c < q.nlim) {
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<uint4 *>(w + lane * 64 + ((i ^ ((lane >> 1) & 3)) * 16)) =
                                    make_uint4(pack_bf16(acc[16 * c + 4 * i]), pack_bf16(acc[16 * c + 4 * i + 1]),
                                               pack_bf16(acc[16 * c + 4 * i + 2]), pack_bf16(acc[16 * c + 4 * i + 3]));
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(w + (8 * i + r8) * 64 + ((quad ^ ((r8 >> 1) & 3)) * 16));
                                if (m1 + 8 * i + r8 < q.mlim && c0 + 32 * c + 8 * quad < q.nlim)
                                    *reinterpret_cast<uint4 *>(o + (int64_t)(8 * i) * g.N + 32 * c) = v;
                            }
                        }
                    }
                } else {
                    unsigned char *w = outs + warp * kStageOut;
                    float *o = static_cast<float *>(g.out) + (int64_t)(q.m0 + m1 + r8) * g.N + q.n0 + c0 + 4 * quad;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if (c0 + 16 * c < q.nlim) {
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<float4 *>(w + lane * 64 + ((i ^ ((lane >> 1) & 3)) * 16)) =
                                    make_float4(acc[8 * c + 2 * i].x, acc[8 * c + 2 * i].y, acc[8 * c + 2 * i + 1].x, acc[8 * c + 2 * i + 1].y);
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 v = *reinterpret_cast<const float4 *>(w + (8 * i + r8) * 64 + ((quad ^ ((r8 >> 1) & 3)) * 16));
                                if (m1 + 8 * i + r8 < q.mlim) *reinterpret_cast<float4 *>(o + (int64_t)(8 * i) * g.N + 16 * c) = v;
                            }
                        }
                    }
                }
            } else if (MODE == kGrad) {
                // four lanes store 32 neighbouring bytes of a row
                float *o = static_cast<float *>(g.out) + ((int64_t)(g.seg0 + q.seg) * g.N + q.m0 + m1 + r8) * g.K + q.n0 + c0 + 2 * quad;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (m1 + 16 * h + 8 * r + r8 < q.mlim) {
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (c0 + 8 * j < q.nlim)
                                    *reinterpret_cast<float2 *>(o + (int64_t)(16 * h + 8 * r) * g.K + 8 * j) = acc[(h * 16 + j) * 2 + r];
                        }
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (CG == 2) tc::cluster_sync();               // nothing of the neighbour's is in flight here any more
    if (warp == kSumWarps + 1) tc::tmem_free<CG>(tmem_slot, kTmemCols);
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

// Tiles of g.nt columns over CTA groups of CG, for the segments from seg0 on.
template <int MODE, int CG>
cudaError_t run_experts(GemmArgs g, int nseg, const int32_t *seg_off, const int32_t *seg_w, const CUtensorMap &mm,
                        const CUtensorMap &mn, cudaStream_t st) {
    g.stage_bytes = kABytes + (uint32_t)(g.nt / CG) * kKB;
    g.stages = std::min<int>(kMaxStages, (int)(kRingBytes / g.stage_bytes));
    const size_t smem = (size_t)g.stages * g.stage_bytes;
    cudaError_t e = ensure_smem((const void *)k_experts<MODE, CG>, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    for (int s0 = 0; s0 < nseg; s0 += kSegCap) {
        g.nseg = std::min(kSegCap, nseg - s0);
        g.seg0 = s0;
        g.seg_off = seg_off + s0;
        g.seg_w = seg_w ? seg_w + s0 : nullptr;
        if ((e = cudaLaunchKernelEx(&cfg, k_experts<MODE, CG>, mm, mn, g)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_expert_gemm(int nseg, int64_t rows, int n_w, int N, int K, const uint8_t *a, const float *a_scale,
                               const int32_t *seg_off, const int32_t *seg_w, const uint8_t *w, const float *w_scale,
                               void *out, bool bf16, void *ws, cudaStream_t st) {
    GemmArgs g = {};
    g.w_scale = w_scale;
    g.x_scale = a_scale;
    g.out = out;
    g.hdr = ws_at<WsHeader>(ws, 0);
    g.rows = rows;
    g.n_w = n_w;
    g.N = N;
    g.K = K;
    g.KB = (K + kKB - 1) / kKB;
    g.NB = (N + 127) / 128;
    g.out_bf16 = bf16;
    g.vec_scale = g.KB % 4 == 0 && ((uintptr_t)a_scale & 15) == 0;
    // A pair's tile of 256 rows wastes more of a short segment, and two CTAs move
    // their weights with one TMA queue less; 64 experts of N = 2816, K = 4096, rows
    // per expert, one CTA / a pair: 24: 146 / 179 us; 96: 171 / 185; 128: 191 / 201;
    // 192: 239 / 218; 256: 299 / 254
    const bool pair = rows / nseg > 144;
    g.nt = kTileN;
    g.box = kTileM;
    CUtensorMap mx, mw;
    cudaError_t e;
    if ((e = make_map(&mx, a, rows, K, kTileM)) != cudaSuccess) return e;
    if ((e = make_map(&mw, w, (int64_t)n_w * N, K, kTileM)) != cudaSuccess) return e;
    return pair ? run_experts<kProduct, 2>(g, nseg, seg_off, seg_w, mx, mw, st)
                : run_experts<kProduct, 1>(g, nseg, seg_off, seg_w, mx, mw, st);
}

cudaError_t launch_expert_wgrad(int nseg, int64_t rows, int N, int K, int64_t cap, const uint8_t *dy, const float *dy_scale,
                                const uint8_t *x, const float *x_scale, const int32_t *seg_off, float *dw, void *ws,
                                cudaStream_t st) {
    GemmArgs g = {};
    g.seg_all = seg_off;
    g.w_scale = dy_scale;
    g.x_scale = x_scale;
    g.out = dw;
    g.hdr = ws_at<WsHeader>(ws, 0);
    g.rows = rows;
    g.cap = cap;
    g.N = N;
    g.K = K;
    g.nt = kTileN;
    g.box = kTileM;
    CUtensorMap my, mx;
    cudaError_t e;
    if ((e = make_map(&my, dy, N, cap, kTileM)) != cudaSuccess) return e;
    if ((e = make_map(&mx, x, K, cap, g.box)) != cudaSuccess) return e;
    return run_experts<kGrad, 2>(g, nseg, seg_off, nullptr, my, mx, st);
}

}  // namespace topo
