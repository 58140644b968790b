// The experts' matrix products in e4m3 with one float32 scale for each block
// of 128 values along the contraction.
//
//   product   y[r][n]     = sum_b sa[r][b] * sw[e][n / 128][b] * (sum over k in block b of a[r][k] * w[e][n][k])
//             for the rows r of each segment of the dispatch layout, e the segment's weights
//   gradient  dw[i][n][k] = sum_b sdy[b][n] * sx[b][k] * (sum over t in block b of dy[n][t] * x[k][t])
//             b over the 128-row blocks of segment i, dy and x laid out column by column
//
// Tiles of 128 rows (layout rows; the gradient's n) x 256 columns (weight rows;
// the gradient's k).  Persistent CTAs, one per SM, of 12 warps: one streams
// operand tiles with TMA through a ring of shared-memory stages, one issues
// tcgen05.mma (four steps of 32 a block) into tensor memory, two bring the
// scales, and two warpgroups keep the tile's float32 sums in registers, a row x
// 128 columns to a thread, and store them.  Segments start at any row: a tile's
// loads may run past its segment's last row into the next one; those rows are
// computed and not stored.
//
// The product's scales are any float32, so every block leaves tensor memory: it
// is scaled and added to the registers by one packed multiply-add for two
// values, from two accumulators in turn, while the next block is multiplied.
// The row's scale times the weights' is one value per thread and block; the
// scale warps compute them four blocks ahead (a layout row's scales are
// consecutive, so a block's are one line each: loaded by the summing warps
// themselves a block ahead they held them up for the whole latency).
// The gradient's scales are powers of two: the tensor cores apply them
// (kind::mxf8f6f4, a scale for 32 values) and sum in tensor memory, which moves
// to the registers every kFlush blocks, so that no float32 sum runs over more
// than 2048 products.  The scale warps turn each stage's scales into exponents.
//
// What bounds it, on a GB300, per block of 128 x 256 x 128: the tensor core needs
// 512 cycles; operands cross shared memory twice, 96 KB at 128 bytes a cycle,
// 768 cycles; the sums' reads of tensor memory hold the tensor core up for
// 256 more.  The product takes about 1000 cycles a block (690 with the reads
// left out, 800 for the gradient).  Tried: pairs of CTAs (cta_group::2, 256 rows,
// half the column traffic) take 880 cycles for twice the rows, but waste more of
// ragged segments and start slower: equal at 2048 rows a segment, 40 percent
// slower at 128; weights on the rows and layout rows on the columns (no waste on
// ragged segments, a scale per column): slower at every length, 24 rows 163 us
// against 133; reads of 16 lanes instead of 32: 160 cycles more.
// Measured: 131072 rows, N = 4096, K = 7168 over 128 experts: 3.4 ms for a first call,
// 3.6 to 3.8 ms call after call (against the power limit), 2.05 to 2.25 PFLOP/s; 1536 rows, 2816 x 4096, 64 experts: 120 us, 6.3 TB/s; gradient of
// 98304 rows, 2816 x 4096, 64 experts: 1.14 to 1.15 ms, its 2.95 GB of output included
// (0.94 ms without the stores; 1.19 ms when the warps read the turned rows back and
// stored them, against one TMA store of 32 rows x 64 bytes; 16 rows x 128 bytes the
// same).  Tiles of 256 x 192, which the two accumulators fill, kept in tensor memory and
// taken while the next tile is multiplied: 1.20 ms, since each product of 128 rows reads
// its columns again (1088 cycles of shared memory for one and a half times the work).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "tcgen.cuh"

namespace topo {
namespace {

enum { kProduct = 0, kGrad = 1 };

constexpr int kKB = 128;                          // contraction values of a block: one 128-byte swizzle row
constexpr int kTileM = 128;
constexpr int kTileN = 256;
constexpr int kSumWarps = 8;                      // warps that scale, add and store
constexpr int kThreads = (kSumWarps + 4) * 32;    // two summing warpgroups, one of producer, issuer and two scale warps
// registers of a thread of the summing and of the other warpgroup; 2 * 128 times
// the one and 128 times the other are the launch's share, 384 * 168
template <int MODE>
constexpr int kSumRegs = MODE == kProduct ? 224 : 208;
template <int MODE>
constexpr int kIoRegs = (384 * 168 - 256 * kSumRegs<MODE>) / 128;
constexpr int kTmemCols = 512;                    // two accumulators of 256 columns, or one and the scales
constexpr uint32_t kABytes = kTileM * kKB;
constexpr int kStages = 4;                        // 48 KB of operands each
static_assert(kStages % 2 == 0, "the two scale warps take the stages in turn, and each keeps its own: the barriers' parity repeats");
// Rows up to which a tile loads only them, 16 at a time, not 128: 8 rows of 8
// experts, 4096 x 7168: 62 -> 45 us; 6 of 64, 4096 x 1408: 13.4 -> 11.0; no
// difference where every SM streams weights anyway (24 rows an expert).
constexpr int kFew = 32;
constexpr int kScaleKB = 4;                       // blocks whose scales are brought together
constexpr int kFlush = 16;                        // gradient: blocks summed in tensor memory before the sum
                                                  // moves to registers
template <int MODE>
constexpr int kSegCap = MODE == kProduct ? 1024 : 512;   // segments of one launch (the table in shared memory)
constexpr uint32_t kStageOut = 2048;              // bytes a warp stores through shared memory at a time
constexpr int kSms = 152;
constexpr int kMostTiles = 1 << 30;               // of one launch; segments in order have fewer than 2^26

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

template <int MODE>
__device__ __forceinline__ int tiles_of(const GemmArgs &g, int len) {
    const int m = MODE == kProduct ? len : g.N, n = MODE == kProduct ? g.N : g.K;
    return ((m + kTileM - 1) / kTileM) * ((n + kTileN - 1) / kTileN);
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
    const int me = MODE == kProduct ? len : g.N, ne = MODE == kProduct ? g.N : g.K;
    const int nm = (me + kTileM - 1) / kTileM, n = loc / nm, m = loc - n * nm;
    r.w = MODE == kGrad ? 0 : g.seg_w ? __ldg(g.seg_w + lo) : g.seg0 + lo;
    r.m0 = m * kTileM;
    r.mlim = min(kTileM, me - r.m0);
    r.n0 = n * kTileN;
    r.nlim = min(kTileN, ne - r.n0);
    if (MODE == kProduct) r.m0 += so[lo];
    r.ncols = (r.nlim + 15) & ~15;
    r.kb0 = MODE == kGrad ? pad[lo] : 0;
    // a segment whose blocks the operands do not hold is empty
    r.nkb = MODE != kGrad ? g.KB : pad[lo + 1] <= (int)(g.cap / kKB) ? pad[lo + 1] - pad[lo] : 0;
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Sums of a thread: acc[i] holds columns 2 i and 2 i + 1 of row `lane`.
using Acc = float2[64];

// acc += s * accumulator, 128 columns of this thread's row.  NC columns are read
// while the NC before them are added.
template <int NC>
__device__ __forceinline__ void add_rows(Acc &acc, uint32_t ta, float s) {
    const float2 s2 = make_float2(s, s);
    uint32_t v[2][NC];
    tc::tmem_ld_rows(ta, v[0]);
    tc::tmem_wait(v[0]);
#pragma unroll
    for (int c = 0; c < 128 / NC; ++c) {
        const bool more = c + 1 < 128 / NC;
        if (more) tc::tmem_ld_rows(ta + NC * (c + 1), v[(c + 1) & 1]);
#pragma unroll
        for (int i = 0; i < NC / 2; ++i)
            tc::fma2(acc[NC / 2 * c + i], make_float2(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1])), s2);
        if (more) tc::tmem_wait(v[(c + 1) & 1]);
    }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
k_experts(const __grid_constant__ CUtensorMap map_m, const __grid_constant__ CUtensorMap map_few,
          const __grid_constant__ CUtensorMap map_n, GemmArgs g) {
    extern __shared__ __align__(1024) unsigned char ring[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], scaled[kStages], drained;
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], sc_full[2], sc_empty[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int expired;
    __shared__ int so[kSegCap<MODE> + 1], tp[kSegCap<MODE> + 1], pad[MODE == kGrad ? kSegCap<MODE> + 1 : 1];
    // product: scales of the rows times the weight scale of each half of the columns
    __shared__ float cs[MODE == kProduct ? 2 : 1][kScaleKB][MODE == kProduct ? kTileN : 1];
    __shared__ __align__(1024) unsigned char outs[kSumWarps * kStageOut];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = blockIdx.x, step = gridDim.x;

    if (warp == kSumWarps + 1) tc::tmem_alloc(&tmem_slot, kTmemCols);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&scaled[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&acc_full[b], 1);
            tc::mbar_init(&acc_empty[b], kSumWarps);
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
    pdl_trigger();
    pdl_wait();                                    // everything read or written from here on
    // the segments' row offsets, then the exclusive prefix of their tile counts;
    // a segment outside the layout or without weights has no tiles and is reported.
    // Offsets out of order can make the good segments overlap, any number of times:
    // the sums stop at kMostTiles, and at one block more than the operands hold
    for (int i = tid; i <= g.nseg; i += kThreads) so[i] = __ldg(g.seg_off + i);
    __syncthreads();
    if (warp == 0) {
        int run = 0, prun = 0;
        const int lim = (int)g.rows, cap = (int)(g.cap / kKB);
        if (MODE == kGrad) {                                // blocks of the segments of earlier launches
            for (int i = lane; i < g.seg0; i += 32) {
                const int a = __ldg(g.seg_all + i), b = __ldg(g.seg_all + i + 1);
                if (a >= 0 && b >= a && b <= lim) prun = min(prun + (b - a + kKB - 1) / kKB, cap + 1);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) prun = min(prun + __shfl_xor_sync(0xffffffffu, prun, o), cap + 1);
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
                if (MODE == kProduct && ok && b > a && run > kMostTiles) {
                    set_error(g.hdr, TOPO_ESTATE);
                    ok = false;
                }
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
                    pad[i] = prun + y - pb;
                    if (i == g.nseg - 1) pad[g.nseg] = prun + y;
                }
            }
            run += __shfl_sync(0xffffffffu, x, 31);
            prun = min(prun + __shfl_sync(0xffffffffu, y, 31), cap + 1);
        }
        if (lane == 0) tp[g.nseg] = run;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();

    if (warp >= kSumWarps) {
        tc::regs_dec<kIoRegs<MODE>>();
        const uint32_t tmem = tmem_slot;
        const int ntiles = tp[g.nseg];
        if (warp == kSumWarps) {
            // --------------------------------------------------------- producer
            int s = 0, fill = 0;                       // stage, and how often the ring went round
            bool ok = true;
            for (int t = first; t < ntiles && ok; t += step) {
                const Tile q = find_tile<MODE>(g, tp, so, pad, t);
                const int ym = q.m0;
                const int yn = (MODE == kProduct ? q.w * g.N : 0) + q.n0;
                const int boxes = (q.ncols + kTileM - 1) / kTileM;          // 128 columns to a load
                // few rows: only they are loaded, 16 at a time (what the other rows of the
                // stage hold goes into sums that are not stored)
                const int few = MODE == kProduct && q.mlim <= kFew ? (q.mlim + 15) / 16 : 0;
                uint32_t bytes = (few ? (uint32_t)few * 16 * kKB : kABytes) + (uint32_t)(boxes * kTileM) * kKB;
                // gradient: the scales of the tile's rows and columns, whole pieces of 16
                const uint32_t ms = MODE == kGrad ? 4u * (uint32_t)q.mlim : 0u, ns = MODE == kGrad ? 4u * (uint32_t)q.nlim : 0u;
                bytes += ms + ns;
                for (int kb = 0; kb < q.nkb; ++kb) {
                    if (fill > 0 && !tc::mbar_wait(&empty[s], (uint32_t)(fill - 1) & 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = tc::smem_u32(&full[s]);
                    const uint32_t a = tc::smem_u32(ring) + (uint32_t)s * g.stage_bytes, b = a + kABytes;
                    const int x = (q.kb0 + kb) * kKB;
                    if (tc::elect()) {
                        tc::mbar_expect_tx(bar, bytes);
                        if (few)
                            for (int c = 0; c < few; ++c) tc::tma_load(a + (uint32_t)(c * 16) * kKB, &map_few, x, ym + 16 * c, bar);
                        else
                            tc::tma_load(a, &map_m, x, ym, bar);
                        for (int c = 0; c < boxes; ++c)
                            tc::tma_load(b + (uint32_t)(c * kTileM) * kKB, &map_n, x, yn + c * kTileM, bar);
                        if (MODE == kGrad) {
                            const uint32_t sf = b + kTileN * kKB;
                            tc::bulk_load(sf, g.w_scale + (int64_t)(q.kb0 + kb) * g.N + q.m0, ms, bar);
                            tc::bulk_load(sf + 512, g.x_scale + (int64_t)(q.kb0 + kb) * g.K + q.n0, ns, bar);
                        }
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        ++fill;
                    }
                }
            }
            if (!ok) atomicExch(&expired, 1);
            // loads in flight land before the CTA ends
            for (int i = 0; i < kStages; ++i) {
                const int n = fill + (i < s ? 1 : 0);          // fills of stage i
                if (n > 0 && !tc::mbar_wait(&full[i], (uint32_t)(n - 1) & 1u)) atomicExch(&expired, 1);
            }
        } else if (warp == kSumWarps + 1) {
            // ----------------------------------------------------------- issuer
            int s = 0, fill = 0, it = 0;               // it: accumulators handed on
            bool ok = true;
            for (int t = first; t < ntiles && ok; t += step) {
                const Tile q = find_tile<MODE>(g, tp, so, pad, t);
                const uint32_t idesc = MODE == kGrad ? tc::idesc_scaled(kTileM, q.ncols) : tc::idesc_e4m3(kTileM, q.ncols);
                for (int kb = 0; kb < q.nkb; ++kb) {
                    // the product hands a block on in turn in two accumulators, the gradient
                    // kFlush blocks in one
                    const int b = MODE == kGrad ? 0 : it & 1, round = MODE == kGrad ? it : it >> 1;
                    const bool begin = MODE != kGrad || kb % kFlush == 0;
                    const bool end = MODE != kGrad || kb % kFlush == kFlush - 1 || kb + 1 == q.nkb;
                    if ((begin && round > 0 && !tc::mbar_wait(&acc_empty[b], (uint32_t)(round - 1) & 1u)) ||
                        !tc::mbar_wait(MODE == kGrad ? &scaled[s] : &full[s], (uint32_t)fill & 1u)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t a = tc::smem_u32(ring) + (uint32_t)s * g.stage_bytes;
                    if (tc::elect()) {
                        const uint64_t dm = tc::smem_desc(a), dn = tc::smem_desc(a + kABytes);
                        if (MODE == kGrad) {
                            const uint32_t ts = tmem + kTileN + 16u * (uint32_t)s;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                tc::mma_scaled(tmem, dm + 2 * j, dn + 2 * j, idesc, ts, ts + 4, !begin || j > 0);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)        // 32 bytes on within the swizzled row
                                tc::mma_e4m3(tmem + (uint32_t)(b * kTileN), dm + 2 * j, dn + 2 * j, idesc, j > 0);
                        }
                        tc::mma_commit(tc::smem_u32(&empty[s]));
                        if (end) tc::mma_commit(tc::smem_u32(&acc_full[b]));
                    }
                    __syncwarp();
                    it += end;
                    if (++s == kStages) {
                        s = 0;
                        ++fill;
                    }
                }
            }
            if (tc::elect()) tc::mma_commit(tc::smem_u32(&drained));
            __syncwarp();
            if (!tc::mbar_wait(&drained, 0)) ok = false;
            if (!ok) atomicExch(&expired, 1);
        } else if (warp >= kSumWarps + 2) {
            // ----------------------------------------------------------- scales
            const int sl = tid - (kSumWarps + 2) * 32;           // 0 .. 63
            int gi = 0, s = 0, fill = 0, it = 0;
            bool ok = true;
            for (int t = first; t < ntiles && ok; t += step) {
                const Tile q = find_tile<MODE>(g, tp, so, pad, t);
                const int m1 = q.m0;
                if constexpr (MODE == kGrad) {
                    // the warps take the stages in turn: the loaded scales, powers of two, become
                    // their exponents, four times over (a step of 32 takes one), in the order
                    // of tc::copy_scales, and go to the stage's own tensor-memory columns
                    for (int kb = 0; kb < q.nkb; ++kb, ++it) {
                        if ((it & 1) == (warp & 1)) {
                            ok = tc::mbar_wait(&full[s], (uint32_t)fill & 1u);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            const uint32_t at = (uint32_t)s * g.stage_bytes + kABytes + kTileN * kKB;
                            uint32_t *sf = reinterpret_cast<uint32_t *>(ring + at);
                            uint32_t v[12];
#pragma unroll
                            for (int i = 0; i < 12; ++i) v[i] = ((sf[32 * i + lane] >> 23) & 0xffu) * 0x01010101u;
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 3; ++i)
                                reinterpret_cast<uint4 *>(sf)[32 * i + lane] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                            tc::fence_async();
                            __syncwarp();
                            if (tc::elect()) {
                                const uint32_t ts = tmem + kTileN + 16u * (uint32_t)s, from = tc::smem_u32(ring) + at;
#pragma unroll
                                for (int i = 0; i < 3; ++i) tc::copy_scales(ts + 4 * i, from + 512 * i);
                                tc::mma_commit(tc::smem_u32(&scaled[s]));
                            }
                            __syncwarp();
                        }
                        if (++s == kStages) {
                            s = 0;
                            ++fill;
                        }
                    }
                } else
                for (int kb = 0; kb < q.nkb; kb += kScaleKB, ++gi) {
                    const int slot = gi & 1, nk = min(kScaleKB, q.nkb - kb);
                    float v[2][kScaleKB], w[2][kScaleKB];
                    // weight scales of the two halves of the columns, scales of two rows
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int nb = min(q.n0 / 128 + h, g.NB - 1), row = sl + 64 * h;
                        const float *wp = g.w_scale + ((int64_t)q.w * g.NB + nb) * g.KB + kb;
                        const float *p = g.x_scale + (int64_t)(m1 + row) * g.KB + kb;
                        const bool in = row < q.mlim;
#pragma unroll
                        for (int u = 0; u < kScaleKB; ++u) {
                            w[h][u] = u < nk ? __ldg(wp + u) : 0.f;
                            v[h][u] = 0.f;
                        }
                        if (in && g.vec_scale) {
                            const float4 f = __ldg(reinterpret_cast<const float4 *>(p));
                            v[h][0] = f.x;
                            v[h][1] = f.y;
                            v[h][2] = f.z;
                            v[h][3] = f.w;
                        } else if (in) {
#pragma unroll
                            for (int u = 0; u < kScaleKB; ++u)
                                if (u < nk) v[h][u] = __ldg(p + u);
                        }
                    }
                    if (gi >= 2) ok = tc::mbar_wait(&sc_empty[slot], (uint32_t)((gi >> 1) - 1) & 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int u = 0; u < kScaleKB; ++u) {
                            cs[slot][u][sl + 64 * h] = v[h][u] * w[0][u];
                            cs[slot][u][128 + sl + 64 * h] = v[h][u] * w[1][u];
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
        const uint32_t done = tc::smem_u32(&acc_empty[0]);
        int it = 0, gi = 0;
        bool live = true;
        // an expired wait lets these warps run on without waiting (and without
        // storing), so that they reach the end with the rest of the CTA
        for (int t = first; t < ntiles; t += step) {
            int nkb, ncol;
            {
                const Tile q = find_tile<MODE>(g, tp, so, pad, t);
                nkb = q.nkb;
                // columns of this half; none for a warp whose rows all lie past the tile's
                ncol = wq * 32 < q.mlim ? max(0, min(128, q.ncols - c0)) : 0;
            }
            Acc acc;
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
            constexpr int kStep = MODE == kGrad ? kFlush : 1;
            for (int kb = 0; kb < nkb; kb += kStep, ++it) {
                const int b = MODE == kGrad ? 0 : it & 1, round = MODE == kGrad ? it : it >> 1;
                const int u = kb & (kScaleKB - 1), slot = gi & 1;
                float scale = 1.f;
                if (MODE == kProduct) {
                    if (live && u == 0) live = tc::mbar_wait_tries(&sc_full[slot], (uint32_t)(gi >> 1) & 1u);
                    scale = cs[MODE == kProduct ? slot : 0][u][MODE == kProduct ? c0 + wq * 32 + lane : 0];
                }
                if (live) live = tc::mbar_wait_tries(&acc_full[b], (uint32_t)round & 1u);
                __syncwarp();
                tc::fence_after();
                if (ncol > 0) add_rows<MODE == kProduct ? 32 : 16>(acc, tmem + lanes + (uint32_t)(b * kTileN + c0), scale);
                tc::fence_before();
                __syncwarp();
                const bool last = MODE == kProduct && (u == kScaleKB - 1 || kb + 1 == nkb);
                if (lane == 0) {
                    tc::mbar_arrive(done + 8 * b);
                    if (last) tc::mbar_arrive(tc::smem_u32(&sc_empty[slot]));
                }
                gi += last;
            }
            live = __all_sync(0xffffffffu, live);
            if (!live) continue;
            // found again rather than kept in registers over the loop
            const Tile q = find_tile<MODE>(g, tp, so, pad, t);
            const int m1 = wq * 32;         // this warp's first row, from m0
            // 32 rows x 64 bytes at a time, turned through shared memory so that four lanes
            // store 64 neighbouring bytes: 16-byte pieces, piece index XOR (row / 2)
            unsigned char *w = outs + warp * kStageOut;
            const int swz = (lane >> 1) & 3;
            const int64_t ld = g.N, at = (int64_t)(q.m0 + m1 + r8) * ld + q.n0 + c0;
            if constexpr (MODE == kGrad) {
                // the same 64-byte rows, XOR included, as one TMA store; rows and columns
                // past the segment's end are left out
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (c0 + 16 * c < q.nlim && m1 < q.mlim) {
                        if (tc::elect()) tc::bulk_wait_read();      // the piece before has left shared memory
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<float4 *>(w + lane * 64 + (i ^ swz) * 16) =
                                make_float4(acc[8 * c + 2 * i].x, acc[8 * c + 2 * i].y, acc[8 * c + 2 * i + 1].x, acc[8 * c + 2 * i + 1].y);
                        tc::fence_async();
                        __syncwarp();
                        if (tc::elect()) tc::tma_store(&map_few, q.n0 + c0 + 16 * c, q.m0 + m1, g.seg0 + q.seg, tc::smem_u32(w));
                        __syncwarp();
                    }
                }
            } else if (g.out_bf16) {
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(g.out) + at + 8 * quad;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c0 + 32 * c < q.nlim) {
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4 *>(w + lane * 64 + (i ^ swz) * 16) =
                                make_uint4(pack_bf16(acc[16 * c + 4 * i]), pack_bf16(acc[16 * c + 4 * i + 1]),
                                           pack_bf16(acc[16 * c + 4 * i + 2]), pack_bf16(acc[16 * c + 4 * i + 3]));
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(w + (8 * i + r8) * 64 + ((quad ^ ((r8 >> 1) & 3)) * 16));
                            if (m1 + 8 * i + r8 < q.mlim && c0 + 32 * c + 8 * quad < q.nlim)
                                *reinterpret_cast<uint4 *>(o + (int64_t)(8 * i) * ld + 32 * c) = v;
                        }
                    }
                }
            } else {
                float *o = static_cast<float *>(g.out) + at + 4 * quad;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (c0 + 16 * c < q.nlim) {
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<float4 *>(w + lane * 64 + (i ^ swz) * 16) =
                                make_float4(acc[8 * c + 2 * i].x, acc[8 * c + 2 * i].y, acc[8 * c + 2 * i + 1].x, acc[8 * c + 2 * i + 1].y);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 v = *reinterpret_cast<const float4 *>(w + (8 * i + r8) * 64 + ((quad ^ ((r8 >> 1) & 3)) * 16));
                            if (m1 + 8 * i + r8 < q.mlim) *reinterpret_cast<float4 *>(o + (int64_t)(8 * i) * ld + 16 * c) = v;
                        }
                    }
                }
            }
        }
        if (MODE == kGrad && tc::elect()) tc::bulk_wait();
        if (!live) atomicExch(&expired, 1);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kSumWarps + 1) tc::tmem_free(tmem_slot, kTmemCols);
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

// Map of out[nseg][N][K] in float32, stored in boxes of 32 rows x 16 columns from
// 64-byte rows in the 64-byte swizzle.
cudaError_t make_out_map(CUtensorMap *m, float *out, int nseg, int N, int K) {
    const EncodeFn f = encode_fn();
    if (!f) return cudaErrorNotSupported;
    const cuuint64_t dim[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)nseg};
    const cuuint64_t stride[2] = {(cuuint64_t)K * 4, (cuuint64_t)N * K * 4};
    const cuuint32_t box[3] = {16, 32, 1}, es[3] = {1, 1, 1};
    const CUresult r = f(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, out, dim, stride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MODE>
cudaError_t run_experts(GemmArgs g, int nseg, const int32_t *seg_off, const int32_t *seg_w, const CUtensorMap &mm,
                        const CUtensorMap &mf, const CUtensorMap &mn, cudaStream_t st) {
    // the gradient's stages also hold their scales, and stay on 1024-byte boundaries
    g.stage_bytes = kABytes + (uint32_t)kTileN * kKB + (MODE == kGrad ? 2048 : 0);
    const size_t smem = (size_t)kStages * g.stage_bytes;
    cudaError_t e = ensure_smem((const void *)k_experts<MODE>, smem);
    if (e != cudaSuccess) return e;
    for (int s0 = 0; s0 < nseg; s0 += kSegCap<MODE>) {
        g.nseg = std::min(kSegCap<MODE>, nseg - s0);
        g.seg0 = s0;
        g.seg_off = seg_off + s0;
        g.seg_w = seg_w ? seg_w + s0 : nullptr;
        if ((e = launch_pdl(k_experts<MODE>, dim3(kSms), dim3(kThreads), smem, st, mm, mf, mn, g)) != cudaSuccess) return e;
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
    CUtensorMap mx, mf, mw;
    cudaError_t e;
    if ((e = make_map(&mx, a, rows, K, kTileM)) != cudaSuccess) return e;
    if ((e = make_map(&mf, a, rows, K, 16)) != cudaSuccess) return e;
    if ((e = make_map(&mw, w, (int64_t)n_w * N, K, kTileM)) != cudaSuccess) return e;
    return run_experts<kProduct>(g, nseg, seg_off, seg_w, mx, mf, mw, st);
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
    CUtensorMap my, mx, mo;
    cudaError_t e;
    if ((e = make_map(&my, dy, N, cap, kTileM)) != cudaSuccess) return e;
    if ((e = make_map(&mx, x, K, cap, kTileM)) != cudaSuccess) return e;
    if ((e = make_out_map(&mo, dw, nseg, N, K)) != cudaSuccess) return e;
    return run_experts<kGrad>(g, nseg, seg_off, nullptr, my, mo, mx, st);
}

}  // namespace topo
