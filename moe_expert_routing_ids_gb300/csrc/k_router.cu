// Routing to experts: scores, expert groups, top-k and weights; and the
// gradient of the weights in the logits.
//
//   s = softmax(x) or 1 / (1 + exp(-x)), every operation rounded to float32
//   c = s + bias; without a bias and with one value per group score, x itself
//       (the same order, without the ties that rounding makes); -inf where x
//       is -inf
//   a group's score is the sum of its one or two largest c; the topk_group
//   groups of the largest scores stay
//   ids = the k largest c of the experts that stay, in descending order; equal
//   values go to the lower index, NaN ranks below every number
//   weight_j = scale * s_j / sum s_j over the k chosen, or scale * s_j
//
// A group of G lanes per token, VPL scores to a lane, each logit read once.
// What decides the choice are the rounded c, but few of them matter, so the
// sigmoid is first taken from the hardware's exp2 and reciprocal:
//   - the k-th largest of the lanes' maxima bounds the k-th largest value from
//     below; what reaches it, less a margin for the approximation, is a
//     candidate (10 to 15 of them for k = 8 or 10);
//   - candidates are evaluated as defined and ranked by counting;
//   - groups whose scores are closer than the margin: the row is done again with
//     every score as defined;
//   - rows with NaN or infinities (where groups or the sigmoid are involved; a bias
//     of 3e30 and more, or NaN: every row), many ties: exact_token, which is not for
//     speed (19 rows of 65536 sent there for their groups cost 24 us, its code being
//     read from memory).
// Measured, 1M x 512 softmax, k = 10: 554 us, 4.0 TB/s (weights that are not
// renormalised: 636); 65536 x 256 sigmoid, 4 of 8 groups, k = 8: 44 us, and 56 to 60
// where one of the rows has more than 64 candidates and goes to exact_token (5 draws of
// 40); softmax with a bias, every row by exact_token: 65536 x 256, k = 8: 248 us.
// Bound by the instructions' latency at 24 to 32 warps an SM, 60 to 70 percent of the
// issue slots used: 700 instructions for two rows of 512, 890 for two of 256 in groups.
// The margin: exp2 of a rounded argument is off by |x| 2^-23 + 2^-22 relative,
// times s (1 - s) in s (|x| s (1 - s) < 0.23), the sum and the reciprocal by
// 2^-22 s: 3.3e-7 at most, and the score as defined, rounded four times, by
// 2.5e-7; twice their sum and the roundings of the sums with the bias stay below
// kMargin + |c| kMarginRel.  A group's score a + b is off by what its two values are
// (1.2e-6 and an ulp of each: 1.2e-7 (|a| + |b|), which may cancel in a + b) and the
// sums' own roundings: below kMargin + (|a| + |b|) kMarginRel to either side, so each
// group has bounds of its own, and two groups whose bounds overlap may be in either
// order.
// The row's sum of weights that are not renormalised takes that exp2 of x - max as
// well: a term is off by 2^-22 + |x - max| 2^-22 of itself, at most 2^-22 of the sum's
// largest term each (max of (1 + d) exp(-d) is 1).  The chosen experts' own exp is expf.
#include <cuda_runtime.h>

#include "common.cuh"

namespace topo {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteCand = 64;              // candidates per token before exact_token takes over
constexpr float kMargin = 2e-6f, kMarginRel = 5e-7f;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ bool above(float a, int ia, float b, int ib) {
    const bool na = a != a, nb = b != b;
    if (na != nb) return nb;
    if (!na && a != b) return a > b;
    return ia < ib;
}

// Order key of a score that is not NaN and its expert: larger ranks above.
__device__ __forceinline__ unsigned long long key_of(float v, int e) {
    uint32_t bits = __float_as_uint(v);
    if (bits == 0x80000000u) bits = 0u;
    const uint32_t k32 = (bits & 0x80000000u) ? ~bits : (bits | 0x80000000u);
    return ((unsigned long long)k32 << 32) | (uint32_t)~e;
}

__device__ __forceinline__ float sigmoid_rn(float x) { return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-x))); }

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float sigmoid_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_approx(x * -1.4426950408889634f)));
    return r;
}

// Factor that keeps 1 / sum finite and sum normal for scores near underflow; a power
// of two, so that (s * up) * (1 / (sum * up)) has the bits of s * (1 / sum) elsewhere.
// (s / sum cost 4 to 6 percent of the routing, 38 of a small gradient: a division of
// zero, on the lanes without a slot, leaves its short path.)
__device__ __forceinline__ float lift(float sum) { return sum < 5.421010862427522e-20f ? 8.507059173023462e37f : 1.f; }

template <bool BF>
__device__ __forceinline__ float logit(const void *row, int e) {
    if (BF) return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short *>(row) + e) << 16);
    return __ldg(reinterpret_cast<const float *>(row) + e);
}

// Expert of slot u of lane gl: VEC consecutive experts per 16-byte load, the
// loads strided over the lanes; VEC = 1: lane-strided.
template <int G, int VEC>
__device__ __forceinline__ int expert_of(int u, int gl) {
    return ((u / VEC) * G + gl) * VEC + (u % VEC);
}

template <int VPL, int G, bool BF, int VEC, bool FULL>
__device__ __forceinline__ void load_row(const void *row, int E, int gl, float (&x)[VPL]) {
    if (VEC > 1) {
#pragma unroll
        for (int c = 0; c < VPL / VEC; ++c) {
            const int ch = c * G + gl;
            const bool in = FULL || ch * VEC < E;
            if (BF) {
                const uint4 w = in ? __ldg(reinterpret_cast<const uint4 *>(row) + ch) : make_uint4(0, 0, 0, 0);
                const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    x[c * VEC + 2 * h] = __uint_as_float(q[h] << 16);
                    x[c * VEC + 2 * h + 1] = __uint_as_float(q[h] & 0xffff0000u);
                }
            } else {
                const float4 w = in ? __ldg(reinterpret_cast<const float4 *>(row) + ch) : make_float4(0, 0, 0, 0);
                x[c * VEC] = w.x;
                x[c * VEC + 1] = w.y;
                x[c * VEC + 2] = w.z;
                x[c * VEC + 3] = w.w;
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < VPL; ++u) {
            const int e = u * G + gl;
            x[u] = FULL || e < E ? logit<BF>(row, e) : 0.f;
        }
    }
}

template <int G>
__device__ __forceinline__ float group_max(unsigned mask, float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o, G));
    return v;
}

template <int G>
__device__ __forceinline__ float group_sum(unsigned mask, float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o, G);
    return v;
}

// (m1, m2), the two largest so far, with v.  A NaN is passed over.
__device__ __forceinline__ void push2(float &m1, float &m2, float v) {
    m2 = fmaxf(m2, fminf(m1, v));
    m1 = fmaxf(m1, v);
}

// The k-th largest of the lanes' values: bitonic sort, descending.  kmax: this
// lane keeps the larger value, one bit per compare-exchange stage.
template <int G>
__device__ __forceinline__ float kth_largest(unsigned mask, unsigned kmax, float y, int k) {
    int st = 0;
#pragma unroll
    for (int size = 2; size <= G; size <<= 1)
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1, ++st) {
            const float o = __shfl_xor_sync(mask, y, stride, G);
            y = ((kmax >> st) & 1u) ? fmaxf(y, o) : fminf(y, o);
        }
    return __shfl_sync(mask, y, k - 1, G);
}

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    int64_t ntok;
    int E, k, score, n_group, topk_group, group_top, renorm;
    int by_logit;       // c is the logit itself
    int exact;          // every row by exact_token
    int whole;          // weights are not renormalised: the softmax's sum over the row is needed
    int lpg_log;        // log2 of the lanes that find a group's score
    int stash4;         // they can read four experts at a time
    int chunk_group;    // a 16-byte load's experts are of one group
    float scale;
    FastDiv gdiv;       // by the experts of a group
};

// Shared memory of one token group.
struct RouteScratch {
    float *stash;       // [E rounded up] scores by expert
    unsigned long long *keys;   // candidates
    int *ce;            // candidates' experts
    int *sel;           // chosen experts, and their logits (the fast rows of a sigmoid: scores)
    float *sx;
    float *gsc;         // [n_group] groups' scores; the fast rows of a sigmoid: lower bounds
};

// Every score as defined, the groups, and k rounds of an argmax: chosen experts
// to sel, logits to sx; *m and *total of a softmax over the row.
template <int G, bool BF>
__device__ __noinline__ void exact_row(const RouteArgs &g, const void *row, const RouteScratch &w, unsigned gmask, int gl,
                                       float *row_max, float *row_sum) {
    const int E = g.E, gs = E / g.n_group;
    float m = 0.f, total = 0.f;
    if (g.score == TOPO_SCORE_SOFTMAX) {
        m = -kInf;
        for (int e = gl; e < E; e += G) m = fmaxf(m, logit<BF>(row, e));
        m = group_max<G>(gmask, m);
        if (m == -kInf) m = 0.f;                                  // nothing to subtract in a row of -inf
        for (int e = gl; e < E; e += G) total += expf(logit<BF>(row, e) - m);
        total = group_sum<G>(gmask, total);
    }
    *row_max = m;
    *row_sum = total;
#pragma unroll 4
    for (int e = gl; e < E; e += G) {
        const float x = logit<BF>(row, e);
        float c = x;
        if (!g.by_logit) {
            float s;
            if (g.score == TOPO_SCORE_SOFTMAX) s = total == 0.f ? 0.f : __fdiv_rn(expf(x - m), total);
            else s = sigmoid_rn(x);
            c = __fadd_rn(s, g.bias ? __ldg(g.bias + e) : 0.f);
            if (x == -kInf) c = -kInf;
        }
        w.stash[e] = c;
    }
    __syncwarp(gmask);
    unsigned keep = 0xffffffffu;
    if (g.n_group > 1) {
        for (int q = gl; q < g.n_group; q += G) {
            float a = w.stash[q * gs], b = -kInf;
            bool hb = false;                                      // b holds a value
#pragma unroll 4
            for (int i = 1; i < gs; ++i) {
                const float v = w.stash[q * gs + i];
                if (above(v, i, a, -1)) {
                    b = a;
                    a = v;
                    hb = true;
                } else if (!hb || above(v, i, b, -1)) {
                    b = v;
                    hb = true;
                }
            }
            w.gsc[q] = g.group_top == 2 ? __fadd_rn(a, b) : a;
        }
        __syncwarp(gmask);
        keep = 0;
        for (int q = gl; q < g.n_group; q += G) {
            int rank = 0;
            for (int i = 0; i < g.n_group; ++i) rank += i != q && above(w.gsc[i], i, w.gsc[q], q);
            keep |= (unsigned)(rank < g.topk_group) << q;
        }
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) keep |= __shfl_xor_sync(gmask, keep, o, G);
    }
    // k rounds of an argmax; a lane looks its experts over again only when its
    // best one was taken
    unsigned left = 0u;                                           // this lane's experts, at most 32
    for (int e = gl, u = 0; e < E; e += G, ++u)
        left |= (unsigned)(g.n_group == 1 || ((keep >> fast_quot((unsigned)e, g.gdiv)) & 1u)) << u;
    float mv = 0.f;
    int mi = -1;
    bool look = true;
    for (int j = 0; j < g.k; ++j) {
        if (look) {
            mi = -1;
#pragma unroll 4
            for (int e = gl, u = 0; e < E; e += G, ++u) {
                const float v = w.stash[e];
                if (((left >> u) & 1u) && (mi < 0 || above(v, e, mv, mi))) {
                    mv = v;
                    mi = e;
                }
            }
        }
        float bv = mv;
        int bi = mi;
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(gmask, bv, o, G);
            const int oi = __shfl_xor_sync(gmask, bi, o, G);
            if (oi >= 0 && (bi < 0 || above(ov, oi, bv, bi))) {
                bv = ov;
                bi = oi;
            }
        }
        look = bi == mi;
        if (look) {
            left &= ~(1u << (bi / G));
            w.sel[j] = bi;
            w.sx[j] = logit<BF>(row, bi);
        }
    }
    __syncwarp(gmask);
}

// The chosen of one row, every score as defined: ids and weights.
template <int G, bool BF>
__device__ __noinline__ void exact_token(const RouteArgs &g, const void *row, const RouteScratch &w, unsigned gmask, int gl,
                                         int64_t tok) {
    float m, total;
    exact_row<G, BF>(g, row, w, gmask, gl, &m, &total);
    const bool soft = g.score == TOPO_SCORE_SOFTMAX;
    float mc = m;
    if (soft && g.renorm) {                                       // softmax over the chosen logits
        mc = -kInf;
        for (int j = gl; j < g.k; j += G) mc = fmaxf(mc, w.sx[j]);
        mc = group_max<G>(gmask, mc);
        if (mc == -kInf) mc = 0.f;
    }
    float sum = 0.f;
    if (g.renorm) {
        for (int j = gl; j < g.k; j += G) sum += soft ? expf(w.sx[j] - mc) : sigmoid_rn(w.sx[j]);
        sum = group_sum<G>(gmask, sum);
    }
    const float up = lift(sum), inv = 1.f / (sum * up);
    for (int j = gl; j < g.k; j += G) {
        const float v = w.sx[j];
        float s = soft ? expf(v - mc) : sigmoid_rn(v);
        if (soft && !g.renorm) s = total == 0.f ? 0.f : __fdiv_rn(s, total);
        g.ids[tok * g.k + j] = w.sel[j];
        if (g.renorm) s = sum == 0.f ? 0.f : s * up * inv;
        g.weights[tok * g.k + j] = g.scale * s;
    }
}

// FULL: E == G * VPL, every slot of every lane holds an expert.  SIG: c is the
// sigmoid plus the bias; else the logit (or every row is done by exact_token).
template <int VPL, int G, bool BF, int VEC, bool FULL, bool SIG>
__global__ void __launch_bounds__(kRouteThreads, VPL > 16 ? 3 : 4)
k_route_experts(const __grid_constant__ RouteArgs g) {
    constexpr int kGroups = kRouteThreads / G;
    __shared__ __align__(16) unsigned long long keys_[kGroups][kRouteCand];
    __shared__ int ce_[kGroups][kRouteCand];
    __shared__ int sel_[kGroups][kMaxK];
    __shared__ float sx_[kGroups][kMaxK];
    constexpr int kHi = SIG ? TOPO_ROUTE_MAX_GROUPS : 0;          // upper bounds of the groups' scores, behind the lower ones
    __shared__ __align__(16) float gsc_[kGroups][TOPO_ROUTE_MAX_GROUPS + kHi];
    extern __shared__ __align__(16) float dyn[];
    const int lane = threadIdx.x & 31, gl = lane & (G - 1), grp = threadIdx.x / G;
    const unsigned gmask = G == 32 ? 0xffffffffu : (((1u << (G & 31)) - 1u) << (lane & ~(G - 1)));
    const int E = g.E, k = g.k, Ep = (E + 3) & ~3;
    float *sb = dyn;                                              // [Ep] bias
    pdl_trigger();
    pdl_wait();
    const RouteScratch w = {dyn + Ep + grp * Ep, keys_[grp], ce_[grp], sel_[grp], sx_[grp], gsc_[grp]};
    float bias_odd = 0.f;                                         // NaN with a bias whose sums may not be finite
    if (SIG) {
        for (int e = threadIdx.x; e < Ep; e += kRouteThreads) {
            sb[e] = g.bias && e < E ? __ldg(g.bias + e) : 0.f;
            bias_odd = fmaf(sb[e] * 1e8f, 0.f, bias_odd);
        }
        if (__syncthreads_or(bias_odd != 0.f)) bias_odd = kInf * 0.f;
    }
    unsigned in = VPL >= 32 ? 0xffffffffu : (1u << (VPL & 31)) - 1u;    // slots that hold an expert
    if (!FULL) {
        in = 0;
#pragma unroll
        for (int u = 0; u < VPL; ++u) in |= (unsigned)(expert_of<G, VEC>(u, gl) < E) << u;
    }
    unsigned kmax = 0;
    {
        int st = 0;
#pragma unroll
        for (int size = 2; size <= G; size <<= 1)
#pragma unroll
            for (int stride = size >> 1; stride > 0; stride >>= 1, ++st)
                kmax |= (unsigned)(((gl & stride) == 0) == ((gl & size) == 0)) << st;
    }
    const bool grouped = g.n_group > 1;
    const int gs = E / g.n_group;
    int chunk_of[VPL / VEC];                                      // groups of this lane's loads
#pragma unroll
    for (int c = 0; c < VPL / VEC; ++c) chunk_of[c] = (int)fast_quot((unsigned)((c * G + gl) * VEC), g.gdiv) & 31;
    for (int q = gl; q < TOPO_ROUTE_MAX_GROUPS; q += G) w.gsc[q] = w.gsc[kHi + q] = -kInf;   // past n_group: below every group
    __syncwarp(gmask);
    for (int64_t tok = (int64_t)blockIdx.x * kGroups + grp; tok < g.ntok; tok += (int64_t)gridDim.x * kGroups) {
        const void *row = static_cast<const char *>(g.logits) + (size_t)tok * E * (BF ? 2 : 4);
        if (g.exact) {
            exact_token<G, BF>(g, row, w, gmask, gl, tok);
            __syncwarp(gmask);
            continue;
        }
        float c[VPL];
        float odd = bias_odd;                                     // NaN with any NaN or infinity
        unsigned cm;                                              // candidates among this lane's slots
        bool precise = false, unsure;
#pragma unroll 1
        for (;;) {
            load_row<VPL, G, BF, VEC, FULL>(row, E, gl, c);
            if (SIG || grouped) {
#pragma unroll
                for (int u = 0; u < VPL; ++u) odd = fmaf(c[u], 0.f, odd);
            }
            if (SIG && precise) {
#pragma unroll 1
                for (int e = gl; e < E; e += G) w.stash[e] = __fadd_rn(sigmoid_rn(logit<BF>(row, e)), sb[e]);
                __syncwarp(gmask);
#pragma unroll
                for (int u = 0; u < VPL; ++u) {
                    const int e = expert_of<G, VEC>(u, gl);
                    c[u] = FULL || e < E ? w.stash[e] : 0.f;
                }
                __syncwarp(gmask);
            } else if (SIG) {
#pragma unroll
                for (int u = 0; u < VPL; u += (VEC >= 4 ? 4 : 1)) {
                    const int e = expert_of<G, VEC>(u, gl);
                    if (VEC >= 4) {
                        const float4 b = FULL || e < E ? *reinterpret_cast<const float4 *>(sb + e) : make_float4(0, 0, 0, 0);
                        c[u] = sigmoid_approx(c[u]) + b.x;
                        c[u + (VEC >= 4 ? 1 : 0)] = sigmoid_approx(c[u + (VEC >= 4 ? 1 : 0)]) + b.y;
                        c[u + (VEC >= 4 ? 2 : 0)] = sigmoid_approx(c[u + (VEC >= 4 ? 2 : 0)]) + b.z;
                        c[u + (VEC >= 4 ? 3 : 0)] = sigmoid_approx(c[u + (VEC >= 4 ? 3 : 0)]) + b.w;
                    } else {
                        c[u] = sigmoid_approx(c[u]) + (FULL || e < E ? sb[e] : 0.f);
                    }
                }
            }
            unsigned valid = in;
            unsure = odd != 0.f;
            if (grouped) {
#pragma unroll
                for (int u = 0; u < VPL; u += (VEC >= 4 ? 4 : 1)) {
                    const int e = expert_of<G, VEC>(u, gl);
                    if (FULL || e < E) {
                        if (VEC >= 4) *reinterpret_cast<float4 *>(w.stash + e) = make_float4(c[u], c[u + (VEC >= 4 ? 1 : 0)], c[u + (VEC >= 4 ? 2 : 0)], c[u + (VEC >= 4 ? 3 : 0)]);
                        else w.stash[e] = c[u];
                    }
                }
                __syncwarp(gmask);
                // lpg = G / 2^ceil(log2 n_group) lanes to a group; 16 bytes at a time where
                // they fit, each group starting at another piece (its own banks)
                const int q = gl >> g.lpg_log, sub = gl & ((1 << g.lpg_log) - 1);
                float a = -kInf, b = -kInf;
                if (q < g.n_group) {
                    const float *base = w.stash + q * gs;
                    if (g.stash4) {
                        const int n4 = gs >> (2 + g.lpg_log);
                        int i = q % n4;
                        for (int r = 0; r < n4; ++r) {
                            const float4 v = *reinterpret_cast<const float4 *>(base + 4 * (sub + (i << g.lpg_log)));
                            push2(a, b, v.x);
                            push2(a, b, v.y);
                            push2(a, b, v.z);
                            push2(a, b, v.w);
                            if (++i == n4) i = 0;
                        }
                    } else {
                        for (int i = sub; i < gs; i += 1 << g.lpg_log) push2(a, b, base[i]);
                    }
                }
                for (int o = 1; o < 1 << g.lpg_log; o <<= 1) {
                    const float oa = __shfl_xor_sync(gmask, a, o, G), ob = __shfl_xor_sync(gmask, b, o, G);
                    b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                    a = fmaxf(a, oa);
                }
                if (sub == 0 && q < g.n_group) {
                    const float v = g.group_top == 2 ? a + b : a;
                    if (SIG) {
                        const float size = g.group_top == 2 ? fabsf(a) + fabsf(b) : fabsf(a);
                        const float d = precise ? 0.f : kMargin + size * kMarginRel;
                        w.gsc[q] = v - d;
                        w.gsc[kHi + q] = v + d;
                    } else {
                        w.gsc[q] = v;
                    }
                }
                __syncwarp(gmask);
                bool kept = false;
                if (gl < g.n_group) {
                    // groups that may be above this one, itself among them
                    const float v = w.gsc[gl];
                    int may = 0;
                    if (precise) {                                    // equal scores by index
#pragma unroll 1
                        for (int i = 0; i < g.n_group; ++i) may += i == gl || above(w.gsc[i], i, v, gl);
                    } else {
                        for (int i = 0; i < g.n_group; i += 4) {
                            const float4 o = *reinterpret_cast<const float4 *>(w.gsc + kHi + i);
                            may += (o.x >= v) + (o.y >= v) + (o.z >= v) + (o.w >= v);
                        }
                    }
                    kept = may <= g.topk_group;
                }
                const unsigned keep = __ballot_sync(gmask, kept) >> (lane & ~(G - 1) & 31);
                unsure |= __popc(keep) != g.topk_group;               // fewer are sure to stay
                if (VEC == 1 || g.chunk_group) {                      // a load's experts are of one group
                    unsigned out = 0;
#pragma unroll
                    for (int c = 0; c < VPL / VEC; ++c)
                        out |= ((~keep >> chunk_of[c]) & 1u) * (((1u << (VEC & 31)) - 1u) << (c * VEC));
                    valid &= ~out;
                } else {
#pragma unroll
                    for (int u = 0; u < VPL; ++u) {
                        const int e = expert_of<G, VEC>(u, gl);
                        if (!((keep >> (fast_quot((unsigned)e, g.gdiv) & 31)) & 1u)) valid &= ~(1u << u);
                    }
                }
            }
            float top = -kInf;
            if (FULL && !grouped) {
#pragma unroll
                for (int u = 0; u < VPL; ++u) top = fmaxf(top, c[u]);
            } else {
#pragma unroll
                for (int u = 0; u < VPL; ++u)
                    if ((valid >> u) & 1u) top = fmaxf(top, c[u]);
            }
            float thr = kth_largest<G>(gmask, kmax, top, k);
            if (SIG && !precise) thr -= kMargin + fabsf(thr) * kMarginRel;
            cm = 0;
#pragma unroll
            for (int u = 0; u < VPL; ++u) cm |= c[u] >= thr ? 1u << u : 0u;
            cm &= valid;
            unsure = __any_sync(gmask, unsure);
            if (!unsure || precise || __any_sync(gmask, odd != 0.f)) break;
            precise = true;
            __syncwarp(gmask);
        }
        float total = 0.f, m = 0.f;                               // softmax over the row
        if (!SIG && g.whole) {
            m = -kInf;
#pragma unroll
            for (int u = 0; u < VPL; ++u)
                if (FULL || ((in >> u) & 1u)) m = fmaxf(m, c[u]);
            m = group_max<G>(gmask, m);
            if (m == -kInf) m = 0.f;
            // the difference first: a rounded m log2(e) would not cancel, nor hold for every m
#pragma unroll
            for (int u = 0; u < VPL; ++u)
                if (FULL || ((in >> u) & 1u)) total += exp2_approx((c[u] - m) * 1.4426950408889634f);
            total = group_sum<G>(gmask, total);
        }
        const int cn = __popc(cm);
        int incl = cn;
#pragma unroll
        for (int o = 1; o < G; o <<= 1) {
            const int y = __shfl_up_sync(gmask, incl, o, G);
            if (gl >= o) incl += y;
        }
        const int n = __shfl_sync(gmask, incl, G - 1, G);
        if (n < k || n > kRouteCand || unsure) {
            exact_token<G, BF>(g, row, w, gmask, gl, tok);
            __syncwarp(gmask);
            continue;
        }
        for (int off = incl - cn; cm; cm &= cm - 1) w.ce[off++] = expert_of<G, VEC>(__ffs(cm) - 1, gl);
        __syncwarp(gmask);
        // candidates q = gl, gl + G, ..: score as defined, key; mostly one pass
        unsigned long long key = 0;
        float sc = 0.f;
        for (int q = gl; q < n; q += G) {
            const int e = w.ce[q];
            const float v = logit<BF>(row, e);
            const float sv = SIG ? sigmoid_rn(v) : v;
            const unsigned long long kv = key_of(SIG ? __fadd_rn(sv, sb[e]) : v, e);
            w.keys[q] = kv;
            if (q == gl) {
                key = kv;
                sc = sv;
            }
        }
        if (gl == 0 && (n & 1)) w.keys[n] = 0;                    // an odd count reads one more
        __syncwarp(gmask);
        for (int q = gl; q < n; q += G) {
            if (q != gl) {
                key = w.keys[q];
                const float v = logit<BF>(row, (int)~(uint32_t)key);
                sc = SIG ? sigmoid_rn(v) : v;
            }
            int rank = 0;
            for (int j = 0; j < n; j += 2) {
                const ulonglong2 o = *reinterpret_cast<const ulonglong2 *>(w.keys + j);
                rank += (o.x > key) + (o.y > key);
            }
            if (rank < k) {
                w.sel[rank] = (int)~(uint32_t)key;
                w.sx[rank] = sc;
            }
        }
        __syncwarp(gmask);
        // weights: slot j on lane j (k <= 16 here)
        const bool on = gl < k;
        float s = on ? w.sx[gl] : -kInf;
        if (!SIG) {
            if (g.score == TOPO_SCORE_SOFTMAX) {
                if (g.renorm) {                                   // softmax over the chosen logits, the largest first
                    m = w.sx[0];
                    if (m == -kInf) m = 0.f;
                }
                s = on ? expf(s - m) : 0.f;
                if (!g.renorm) s = total == 0.f ? 0.f : s / total;
            } else {
                s = on ? sigmoid_rn(s) : 0.f;
            }
        } else if (!on) {
            s = 0.f;
        }
        if (g.renorm) {
            const float sum = group_sum<G>(gmask, s), up = lift(sum);
            s = sum == 0.f ? 0.f : s * up * (1.f / (sum * up));
        }
        if (on) {
            g.ids[tok * k + gl] = w.sel[gl];
            g.weights[tok * k + gl] = g.scale * s;
        }
        __syncwarp(gmask);                                        // the scratch is free again
    }
}

// ------------------------------------------------------------------ gradient
struct RouteGradArgs {
    const void *logits;
    const int32_t *ids;
    const float *dw;
    void *dx;
    WsHeader *hdr;
    int64_t ntok;
    int E, k, score, renorm;
    float scale;
};

template <bool BF>
__device__ __forceinline__ void put(void *row, int e, float v) {
    if (BF) {
        const uint32_t b = __float_as_uint(v);
        const uint32_t r = (b & 0x7fffffffu) > 0x7f800000u ? 0x7fc0u : (b + 0x7fffu + ((b >> 16) & 1u)) >> 16;
        reinterpret_cast<unsigned short *>(row)[e] = (unsigned short)r;
    } else {
        reinterpret_cast<float *>(row)[e] = v;
    }
}

// One warp per token: the row's dense gradient (0, or -p_e * sum for a softmax
// whose weights are not renormalised), then the chosen experts' values over it.
// Bound by memory: 1M tokens x 512 in 500 us, 2.1 GB written and 10 sectors of 64
// bytes read for each token's chosen logits, 5.8 TB/s (V: the rows are written 16
// bytes at a time, else 579 us; ids and logits of later tokens loaded ahead
// changed nothing).  Dense rows (a softmax that is not renormalised) are read three
// times and written a value at a time: 1050 us.
template <bool BF, bool V>
__global__ void __launch_bounds__(256)
k_route_grad(RouteGradArgs g) {
    const int lane = threadIdx.x & 31;
    const int64_t nw = (int64_t)gridDim.x * (blockDim.x >> 5);
    const int E = g.E, k = g.k;
    const bool soft = g.score == TOPO_SCORE_SOFTMAX, dense = soft && !g.renorm;
    pdl_trigger();
    pdl_wait();
    for (int64_t tok = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); tok < g.ntok; tok += nw) {
        const char *row = static_cast<const char *>(g.logits) + (size_t)tok * E * (BF ? 2 : 4);
        char *out = static_cast<char *>(g.dx) + (size_t)tok * E * (BF ? 2 : 4);
        // slots lane and lane + 32
        int id[2];
        float gr[2], x[2], s[2], w[2];
        bool bad = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = lane + 32 * h;
            id[h] = -1;
            gr[h] = 0.f;
            if (j < k) {
                id[h] = __ldg(g.ids + tok * k + j);
                gr[h] = __ldg(g.dw + tok * k + j);
                if ((unsigned)id[h] >= (unsigned)E) {
                    bad = true;
                    id[h] = -1;
                }
            }
        }
        if (bad) set_error(g.hdr, TOPO_ERANGE);
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h] = id[h] >= 0 ? logit<BF>(row, id[h]) : -kInf;
        if (!dense) {
            if (V) {
                const int nv = E * (BF ? 2 : 4) / 16;
                for (int i = lane; i < nv; i += 32) reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
            } else {
                for (int e = lane; e < E; e += 32) put<BF>(out, e, 0.f);
            }
        }
        float m = -kInf, total = 0.f;
        if (soft) {
            if (g.renorm) m = fmaxf(x[0], x[1]);
            else
                for (int e = lane; e < E; e += 32) m = fmaxf(m, logit<BF>(row, e));
            m = group_max<32>(0xffffffffu, m);
            if (m == -kInf) m = 0.f;
            if (dense) {
                for (int e = lane; e < E; e += 32) total += expf(logit<BF>(row, e) - m);
                total = group_sum<32>(0xffffffffu, total);
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = id[h] < 0 ? 0.f : soft ? expf(x[h] - m) : sigmoid_rn(x[h]);
            sum += s[h];
        }
        if (dense) sum = total;
        else if (g.renorm) sum = group_sum<32>(0xffffffffu, sum);
        else sum = 1.f;
        const float up = lift(sum), inv = sum == 0.f ? 0.f : 1.f / (sum * up);
        float dot = 0.f;                                          // sum of g_j w_j / scale
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = soft || g.renorm ? s[h] * up * inv : s[h];
            dot += gr[h] * w[h];
        }
        dot = soft || g.renorm ? group_sum<32>(0xffffffffu, dot) : 0.f;
        if (dense) {
            const float f = -g.scale * dot * inv;
            for (int e = lane; e < E; e += 32) put<BF>(out, e, f == 0.f ? 0.f : f * expf(logit<BF>(row, e) - m));
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (id[h] >= 0) {
                float d = g.scale * w[h] * (gr[h] - dot);
                // 1 - s = s exp(-x): from the rounded s it would be 0 from 17.4 on
                if (!soft) d *= s[h] == 0.f ? 1.f : s[h] * expf(-x[h]);
                put<BF>(out, id[h], d);
            }
    }
}

template <int VPL, int G, bool BF, int VEC, bool FULL, bool SIG>
cudaError_t run_route(const RouteArgs &a, cudaStream_t st) {
    constexpr int kGroups = kRouteThreads / G;
    const auto fn = k_route_experts<VPL, G, BF, VEC, FULL, SIG>;
    const size_t smem = (size_t)(kGroups + 1) * ((a.E + 3) & ~3) * 4;
    cudaError_t e = ensure_smem((const void *)fn, smem);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.ntok + kGroups - 1) / kGroups;
    const int64_t most = 152 * (VPL > 16 ? 3 : 4);                // the CTAs that run together
    return launch_pdl(fn, dim3((unsigned)(want < most ? want : most)), dim3(kRouteThreads), smem, st, a);
}

template <int VPL, int G, bool BF, int VEC, bool FULL>
cudaError_t route_sig(const RouteArgs &a, cudaStream_t st) {
    if (a.by_logit) return run_route<VPL, G, BF, VEC, FULL, false>(a, st);
    return run_route<VPL, G, BF, VEC, FULL, true>(a, st);
}

template <int VPL, int G, bool BF>
cudaError_t route_vec(RouteArgs a, bool vec, cudaStream_t st) {
    constexpr int V = BF ? 8 : 4;
    constexpr int W = VPL % V == 0 ? V : 1;
    const int gs = a.E / a.n_group;
    a.lpg_log = 0;
    while ((a.n_group << (a.lpg_log + 1)) <= G) ++a.lpg_log;
    a.stash4 = gs % (4 << a.lpg_log) == 0;
    a.chunk_group = gs % W == 0;
    if (W > 1 && vec) {
        if (a.E == G * VPL) return route_sig<VPL, G, BF, W, true>(a, st);
        return route_sig<VPL, G, BF, W, false>(a, st);
    }
    return route_sig<VPL, G, BF, 1, false>(a, st);
}

// 16 lanes per token up to 512 experts (two tokens of a warp share the sort,
// scan and ranking), else 32.
template <bool BF>
cudaError_t route_vpl(const RouteArgs &a, bool vec, cudaStream_t st) {
    if (a.E <= 512) {
        const int vpl = (a.E + 15) / 16;
        if (vpl <= 4) return route_vec<4, 16, BF>(a, vec, st);
        if (vpl <= 8) return route_vec<8, 16, BF>(a, vec, st);
        if (vpl <= 16) return route_vec<16, 16, BF>(a, vec, st);
        return route_vec<32, 16, BF>(a, vec, st);
    }
    return route_vec<32, 32, BF>(a, vec, st);
}

}  // namespace

cudaError_t launch_route(const topo_route_opts &o, int64_t ntok, int E, int k, const void *logits, bool bf16,
                         const float *bias, int32_t *ids, float *weights, cudaStream_t st) {
    RouteArgs a = {};
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.ntok = ntok;
    a.E = E;
    a.k = k;
    a.score = o.score;
    a.n_group = o.n_group;
    a.topk_group = o.topk_group;
    a.group_top = o.group_top;
    a.renorm = o.renorm;
    a.scale = o.scale;
    a.by_logit = !bias && o.group_top == 1;
    // a softmax that the choice needs has no cheap bound; 16 lanes hold the
    // candidates of at most 16 slots and the scores of at most 16 groups
    a.exact = (o.score == TOPO_SCORE_SOFTMAX && !a.by_logit) || k > 16 || o.n_group > 16;
    a.whole = o.score == TOPO_SCORE_SOFTMAX && !o.renorm;
    a.gdiv = make_fast_div((unsigned)(E / o.n_group));
    if (ntok == 0) return cudaSuccess;
    const bool vec = ((uintptr_t)logits & 15) == 0 && ((size_t)E * (bf16 ? 2 : 4)) % 16 == 0;
    return bf16 ? route_vpl<true>(a, vec, st) : route_vpl<false>(a, vec, st);
}

cudaError_t launch_route_grad(const topo_route_opts &o, int64_t ntok, int E, int k, const void *logits, bool bf16,
                              const int32_t *ids, const float *dw, void *dx, void *ws, cudaStream_t st) {
    RouteGradArgs a = {logits, ids, dw, dx, ws_at<WsHeader>(ws, 0), ntok, E, k, o.score, o.renorm, o.scale};
    if (ntok == 0) return cudaSuccess;
    const int64_t want = (ntok + 7) / 8;
    const unsigned blocks = (unsigned)(want < 152 * 32 ? want : 152 * 32);
    const bool v = ((uintptr_t)dx & 15) == 0 && ((size_t)E * (bf16 ? 2 : 4)) % 16 == 0;
    const auto fn = bf16 ? (v ? k_route_grad<true, true> : k_route_grad<true, false>)
                         : (v ? k_route_grad<false, true> : k_route_grad<false, false>);
    return launch_pdl(fn, dim3(blocks), dim3(256), 0, st, a);
}

}  // namespace topo
