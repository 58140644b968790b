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
// A group of G lanes per token, VPL scores to a lane.  The k-th largest of the
// lanes' maxima bounds the k-th largest score from below, so the scores that
// reach it are the only candidates, and a candidate's place is the number of
// candidates above it; rows where that fails (few lanes, many ties, NaN) take
// k rounds of an exact argmax.
#include <cuda_runtime.h>

#include "common.cuh"

namespace topo {
namespace {

constexpr int kRouteThreads = 128;
constexpr int kRouteCand = 64;              // candidates per token before the exact rounds take over
constexpr int kMaxGroups = 32;

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

template <bool BF>
__device__ __forceinline__ float logit(const void *row, int e) {
    if (BF) return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short *>(row) + e) << 16);
    return __ldg(reinterpret_cast<const float *>(row) + e);
}

// Expert of slot u of lane gl: VEC consecutive experts per 16-byte load.
template <int G, int VEC>
__device__ __forceinline__ int expert_of(int u, int gl) {
    return VEC > 1 ? ((u / VEC) * G + gl) * VEC + (u % VEC) : u * G + gl;
}

template <int VPL, int G, bool BF, int VEC>
__device__ __forceinline__ void load_row(const void *row, int E, int gl, float *x) {
    if (VEC > 1) {
#pragma unroll
        for (int c = 0; c < VPL / VEC; ++c) {
            const int ch = c * G + gl;
            const bool in = ch * VEC < E;
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
            x[u] = e < E ? logit<BF>(row, e) : 0.f;
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

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    int64_t ntok;
    int E, k, score, n_group, topk_group, group_top, renorm;
    float scale;
};

template <int VPL, int G, bool BF, int VEC>
__global__ void __launch_bounds__(kRouteThreads)
k_route_experts(RouteArgs g) {
    constexpr int kGroups = kRouteThreads / G;
    __shared__ float stash_[kGroups][G * VPL];
    __shared__ unsigned long long keys_[kGroups][kRouteCand];
    __shared__ int sel_[kGroups][kMaxK];
    __shared__ float gsc_[kGroups][kMaxGroups];
    const int lane = threadIdx.x & 31, gl = lane & (G - 1), grp = threadIdx.x / G;
    const unsigned gmask = G == 32 ? 0xffffffffu : (((1u << (G & 31)) - 1u) << (lane & ~(G - 1)));
    float *stash = stash_[grp], *gsc = gsc_[grp];
    unsigned long long *wk = keys_[grp];
    int *sel = sel_[grp];
    const int E = g.E, k = g.k;
    const bool by_logit = !g.bias && g.group_top == 1;
    unsigned in = 0;                                              // slots that hold an expert
#pragma unroll
    for (int u = 0; u < VPL; ++u) in |= (unsigned)(expert_of<G, VEC>(u, gl) < E) << u;
    // bitonic directions of this lane, one bit per compare-exchange stage
    unsigned kmax = 0;
    {
        int st = 0;
#pragma unroll
        for (int size = 2; size <= G; size <<= 1)
#pragma unroll
            for (int stride = size >> 1; stride > 0; stride >>= 1, ++st)
                kmax |= (unsigned)(((gl & stride) == 0) == ((gl & size) == 0)) << st;
    }
    for (int64_t tok = (int64_t)blockIdx.x * kGroups + grp; tok < g.ntok; tok += (int64_t)gridDim.x * kGroups) {
        const void *row = static_cast<const char *>(g.logits) + (size_t)tok * E * (BF ? 2 : 4);
        float x[VPL], c[VPL];
        load_row<VPL, G, BF, VEC>(row, E, gl, x);
        float m = 0.f, total = 0.f;                               // softmax: row maximum, sum of exp(x - m)
        const bool whole = g.score == TOPO_SCORE_SOFTMAX && (!by_logit || !g.renorm);
        if (whole) {
            m = -kInf;
            bool nan = false;
#pragma unroll
            for (int u = 0; u < VPL; ++u)
                if ((in >> u) & 1u) {
                    m = fmaxf(m, x[u]);
                    nan |= x[u] != x[u];
                }
            m = group_max<G>(gmask, m);
            if (m == -kInf) m = 0.f;                              // nothing to subtract in a row of -inf
#pragma unroll
            for (int u = 0; u < VPL; ++u)
                if ((in >> u) & 1u) total += expf(x[u] - m);
            total = group_sum<G>(gmask, total);
        }
#pragma unroll
        for (int u = 0; u < VPL; ++u) {
            if (by_logit) {
                c[u] = x[u];
            } else {
                float s;
                if (g.score == TOPO_SCORE_SOFTMAX) s = total == 0.f ? 0.f : __fdiv_rn(expf(x[u] - m), total);
                else s = sigmoid_rn(x[u]);
                const int e = expert_of<G, VEC>(u, gl);
                c[u] = __fadd_rn(s, g.bias && e < E ? __ldg(g.bias + e) : 0.f);
                if (x[u] == -kInf) c[u] = -kInf;
            }
        }
        unsigned valid = in;
        if (g.n_group > 1) {
            const int gs = E / g.n_group;
#pragma unroll
            for (int u = 0; u < VPL; ++u) stash[expert_of<G, VEC>(u, gl)] = c[u];
            __syncwarp(gmask);
            for (int q = gl; q < g.n_group; q += G) {
                float a = stash[q * gs], b = -kInf;
                bool hb = false;                                  // b holds a value
                for (int i = 1; i < gs; ++i) {
                    const float v = stash[q * gs + i];
                    if (above(v, i, a, -1)) {
                        b = a;
                        a = v;
                        hb = true;
                    } else if (!hb || above(v, i, b, -1)) {
                        b = v;
                        hb = true;
                    }
                }
                gsc[q] = g.group_top == 2 ? __fadd_rn(a, b) : a;
            }
            __syncwarp(gmask);
            unsigned keep = 0;
            for (int q = gl; q < g.n_group; q += G) {
                int rank = 0;
                for (int i = 0; i < g.n_group; ++i) rank += i != q && above(gsc[i], i, gsc[q], q);
                keep |= (unsigned)(rank < g.topk_group) << q;
            }
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) keep |= __shfl_xor_sync(gmask, keep, o, G);
#pragma unroll
            for (int u = 0; u < VPL; ++u) {
                const int e = expert_of<G, VEC>(u, gl);
                if (e < E && !((keep >> (e / gs)) & 1u)) valid &= ~(1u << u);
            }
        }
        // tau: the k-th largest lane maximum (bitonic sort, descending)
        float tau = -kInf;
        if (k <= G) {
            float y = -kInf;
#pragma unroll
            for (int u = 0; u < VPL; ++u)
                if ((valid >> u) & 1u) y = fmaxf(y, c[u]);
            int st = 0;
#pragma unroll
            for (int size = 2; size <= G; size <<= 1)
#pragma unroll
                for (int stride = size >> 1; stride > 0; stride >>= 1, ++st) {
                    const float o = __shfl_xor_sync(gmask, y, stride, G);
                    y = ((kmax >> st) & 1u) ? fmaxf(y, o) : fminf(y, o);
                }
            tau = __shfl_sync(gmask, y, k - 1, G);
        }
        unsigned cm = 0;
#pragma unroll
        for (int u = 0; u < VPL; ++u) cm |= (unsigned)(((valid >> u) & 1u) && c[u] >= tau) << u;
        const int cn = __popc(cm);
        int incl = cn;
#pragma unroll
        for (int o = 1; o < G; o <<= 1) {
            const int y = __shfl_up_sync(gmask, incl, o, G);
            if (gl >= o) incl += y;
        }
        const int n = __shfl_sync(gmask, incl, G - 1, G);
        if (k <= G && n >= k && n <= kRouteCand) {
            int off = incl - cn;
#pragma unroll
            for (int u = 0; u < VPL; ++u)
                if ((cm >> u) & 1u) wk[off++] = key_of(c[u], expert_of<G, VEC>(u, gl));
            __syncwarp(gmask);
            for (int q = gl; q < n; q += G) {
                const unsigned long long key = wk[q];
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < n; ++j) rank += wk[j] > key;
                if (rank < k) sel[rank] = (int)~(uint32_t)key;
            }
        } else {
            unsigned left = valid;
            for (int j = 0; j < k; ++j) {
                float bv = 0.f;
                int bi = -1;
#pragma unroll
                for (int u = 0; u < VPL; ++u) {
                    const int e = expert_of<G, VEC>(u, gl);
                    if (((left >> u) & 1u) && (bi < 0 || above(c[u], e, bv, bi))) {
                        bv = c[u];
                        bi = e;
                    }
                }
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) {
                    const float ov = __shfl_xor_sync(gmask, bv, o, G);
                    const int oi = __shfl_xor_sync(gmask, bi, o, G);
                    if (oi >= 0 && (bi < 0 || above(ov, oi, bv, bi))) {
                        bv = ov;
                        bi = oi;
                    }
                }
#pragma unroll
                for (int u = 0; u < VPL; ++u)
                    if (expert_of<G, VEC>(u, gl) == bi) left &= ~(1u << u);
                if (gl == 0) sel[j] = bi;
            }
        }
        __syncwarp(gmask);
        // weights of the chosen, slot j on lane j (and j + G, ...)
        float mc = m;
        const bool soft = g.score == TOPO_SCORE_SOFTMAX;
        if (soft && g.renorm) {                                   // softmax over the chosen logits
            mc = -kInf;
            for (int j = gl; j < k; j += G) mc = fmaxf(mc, logit<BF>(row, sel[j]));
            mc = group_max<G>(gmask, mc);
            if (mc == -kInf) mc = 0.f;
        }
        float sum = 0.f;
        if (g.renorm) {
            for (int j = gl; j < k; j += G) {
                const float v = logit<BF>(row, sel[j]);
                sum += soft ? expf(v - mc) : sigmoid_rn(v);
            }
            sum = group_sum<G>(gmask, sum);
        }
        for (int j = gl; j < k; j += G) {
            const int e = sel[j];
            const float v = logit<BF>(row, e);
            float s = soft ? expf(v - mc) : sigmoid_rn(v);
            if (soft && !g.renorm) s = total == 0.f ? 0.f : __fdiv_rn(s, total);
            float w = g.scale * s;
            if (g.renorm) w = sum == 0.f ? 0.f : s * (g.scale / sum);
            g.ids[tok * k + j] = e;
            g.weights[tok * k + j] = w;
        }
        __syncwarp(gmask);                                        // sel, keys and stash are free again
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
template <bool BF>
__global__ void __launch_bounds__(256)
k_route_grad(RouteGradArgs g) {
    const int lane = threadIdx.x & 31;
    const int64_t nw = (int64_t)gridDim.x * (blockDim.x >> 5);
    const int E = g.E, k = g.k;
    const bool soft = g.score == TOPO_SCORE_SOFTMAX;
    for (int64_t tok = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); tok < g.ntok; tok += nw) {
        const char *row = static_cast<const char *>(g.logits) + (size_t)tok * E * (BF ? 2 : 4);
        char *out = static_cast<char *>(g.dx) + (size_t)tok * E * (BF ? 2 : 4);
        // slots lane and lane + 32
        int id[2];
        float gr[2], s[2], w[2];
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
        float m = -kInf, total = 0.f;
        if (soft) {
            if (g.renorm) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (id[h] >= 0) m = fmaxf(m, logit<BF>(row, id[h]));
            } else {
                for (int e = lane; e < E; e += 32) m = fmaxf(m, logit<BF>(row, e));
            }
            m = group_max<32>(0xffffffffu, m);
            if (m == -kInf) m = 0.f;
            if (!g.renorm) {
                for (int e = lane; e < E; e += 32) total += expf(logit<BF>(row, e) - m);
                total = group_sum<32>(0xffffffffu, total);
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = 0.f;
            if (id[h] >= 0) {
                const float x = logit<BF>(row, id[h]);
                s[h] = soft ? expf(x - m) : sigmoid_rn(x);
            }
            sum += s[h];
        }
        if (soft && !g.renorm) sum = total;
        else if (g.renorm) sum = group_sum<32>(0xffffffffu, sum);
        else sum = 1.f;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        float dot = 0.f;                                          // sum of g_j w_j / scale
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = soft || g.renorm ? s[h] * inv : s[h];
            dot += gr[h] * w[h];
        }
        dot = soft || g.renorm ? group_sum<32>(0xffffffffu, dot) : 0.f;
        if (soft && !g.renorm) {
            const float f = -g.scale * dot * inv;
            for (int e = lane; e < E; e += 32) put<BF>(out, e, f == 0.f ? 0.f : f * expf(logit<BF>(row, e) - m));
        } else {
            for (int e = lane; e < E; e += 32) put<BF>(out, e, 0.f);
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (id[h] >= 0) {
                float d = g.scale * w[h] * (gr[h] - dot);
                if (!soft) d *= 1.f - s[h];
                put<BF>(out, id[h], d);
            }
        __syncwarp();
    }
}

template <int VPL, int G, bool BF, int VEC>
cudaError_t run_route(const RouteArgs &a, cudaStream_t st) {
    constexpr int kGroups = kRouteThreads / G;
    const int64_t want = (a.ntok + kGroups - 1) / kGroups;
    const unsigned blocks = (unsigned)(want < 152 * 16 ? want : 152 * 16);
    k_route_experts<VPL, G, BF, VEC><<<blocks, kRouteThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int VPL, int G, bool BF>
cudaError_t route_vec(const RouteArgs &a, bool vec, cudaStream_t st) {
    constexpr int V = BF ? 8 : 4;
    if (vec && VPL % V == 0) return run_route<VPL, G, BF, (VPL % V == 0 ? V : 1)>(a, st);
    return run_route<VPL, G, BF, 1>(a, st);
}

template <bool BF>
cudaError_t route_vpl(const RouteArgs &a, bool vec, cudaStream_t st) {
    if (a.E <= 512 && a.k <= 12) {
        const int vpl = (a.E + 15) / 16;
        if (vpl <= 4) return route_vec<4, 16, BF>(a, vec, st);
        if (vpl <= 8) return route_vec<8, 16, BF>(a, vec, st);
        if (vpl <= 16) return route_vec<16, 16, BF>(a, vec, st);
        return route_vec<32, 16, BF>(a, vec, st);
    }
    const int vpl = (a.E + 31) / 32;
    if (vpl <= 4) return route_vec<4, 32, BF>(a, vec, st);
    if (vpl <= 8) return route_vec<8, 32, BF>(a, vec, st);
    if (vpl <= 16) return route_vec<16, 32, BF>(a, vec, st);
    return route_vec<32, 32, BF>(a, vec, st);
}

}  // namespace

cudaError_t launch_route(const topo_route_opts &o, int64_t ntok, int E, int k, const void *logits, bool bf16,
                         const float *bias, int32_t *ids, float *weights, cudaStream_t st) {
    RouteArgs a = {logits, bias, ids, weights, ntok, E, k, o.score, o.n_group, o.topk_group, o.group_top, o.renorm, o.scale};
    if (ntok == 0) return cudaSuccess;
    const bool vec = ((uintptr_t)logits & 15) == 0 && ((size_t)E * (bf16 ? 2 : 4)) % 16 == 0;
    return bf16 ? route_vpl<true>(a, vec, st) : route_vpl<false>(a, vec, st);
}

cudaError_t launch_route_grad(const topo_route_opts &o, int64_t ntok, int E, int k, const void *logits, bool bf16,
                              const int32_t *ids, const float *dw, void *dx, void *ws, cudaStream_t st) {
    RouteGradArgs a = {logits, ids, dw, dx, ws_at<WsHeader>(ws, 0), ntok, E, k, o.score, o.renorm, o.scale};
    if (ntok == 0) return cudaSuccess;
    const int64_t want = (ntok + 7) / 8;
    const unsigned blocks = (unsigned)(want < 152 * 8 ? want : 152 * 8);
    if (bf16) k_route_grad<true><<<blocks, 256, 0, st>>>(a);
    else k_route_grad<false><<<blocks, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace topo
