// router_grad.cu -- what the router is trained with: the balance loss, the
// gradient of the gate's logits, and the weighted sum's backward pass.
//
// With p = softmax(logits[t]), sequence s of n_s unmasked tokens, c[s, e] the
// assignments of its tokens to expert e, and S+ sequences that have any:
//   prob_mean[s, e] = (1 / n_s) sum_t p[t, e]
//   loss = (coef / S+) sum_s E / (k n_s) sum_e c[s, e] prob_mean[s, e]
// The counts have no gradient, so
//   d loss / d logits[t, i] = coef E / (S+ k n_s^2) p_i (c[s, i] - sum_e p_e c[s, e]),
// and through the chosen weights, with j over the k slots,
//   w_j = p_{i_j} / sum_l p_{i_l}:  d logits[i_j] += w_j (dw_j - sum_l w_l dw_l)
//   w_j = p_{i_j}:  d logits[e] += sum_{j: i_j = e} p_e dw_j - p_e sum_l p_{i_l} dw_l.
//
// Bound: the logits are read once by each pass and the gradient written once;
// in practice the instructions of a row's reductions count as much.  A group of
// 8, 16 or 32 lanes holds a token's row in registers, as few lanes as leave
// each up to 16 values: a reduction over 8 lanes takes three shuffles for four
// tokens, one over 32 takes five for one.  Measured at T = 250007, E = 160, nine
// sequences: partial sums 33 us (160 MB, 4.9 TB/s; 98 instructions a token, the
// issue slots 70% busy), joining them 7 us, gradient 52 us (320 MB, 6.2 TB/s).
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int R_THREADS = 256;
constexpr int R_WARPS = R_THREADS / 32;
constexpr float kNegInf = -__builtin_huge_valf();

// Lane l of a token's LPT lanes holds columns (i * LPT + l) * VEC + v,
// i < NC, v < VEC.
template <int VEC, int LPT, int NC>
struct Row {
    static constexpr int N = VEC * NC;
    static __device__ __forceinline__ int col(int l, int i) {
        return ((i / VEC) * LPT + l) * VEC + i % VEC;
    }
    // columns past E read as `fill`
    static __device__ __forceinline__ void load(const float *row, int E, int l, float fill,
                                                float (&z)[N]) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int e = (c * LPT + l) * VEC;
            if (VEC == 4) {
                float4 v = make_float4(fill, fill, fill, fill);
                if (e < E) v = __ldg(reinterpret_cast<const float4 *>(row + e));
                z[c * 4] = v.x;
                z[c * 4 + 1] = v.y;
                z[c * 4 + 2] = v.z;
                z[c * 4 + 3] = v.w;
            } else {
                z[c] = e < E ? __ldg(row + e) : fill;
            }
        }
    }
    static __device__ __forceinline__ void store(float *row, int E, int l, const float (&z)[N]) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int e = (c * LPT + l) * VEC;
            if (e >= E) continue;
            if (VEC == 4)
                __stcs(reinterpret_cast<float4 *>(row + e),
                       make_float4(z[c * 4], z[c * 4 + 1], z[c * 4 + 2], z[c * 4 + 3]));
            else
                __stcs(row + e, z[c]);
        }
    }
};

template <int LPT>
__device__ __forceinline__ float group_max(float v) {
    if constexpr (LPT == 32) {
        asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
    } else {
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    }
    return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

constexpr float kLog2e = 1.4426950408889634f;
// exp(z - m), off by at most (2.3 |z - m| + 4) 2^-24 of it; 0 below 2^-126.
__device__ __forceinline__ float exp_from(float z, float m) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"((z - m) * kLog2e));
    return r;
}

// z -> e = exp(z - m) in place for U rows; mr = (m, 1 / sum of e), so that the
// probabilities are e * mr.y.  A row with no finite logit has mr.y = 0.
// The difference comes first at every magnitude: with 2^(z log2e - m log2e) in
// one fused step what the rounded m log2e is off by stays in the exponent (128
// and more from |m| = 1.5e9 on: the row's own maximum overflows or vanishes),
// and a slot's exp_from(z, m) * mr.y would carry it too.  The fused step saves
// 0.6 of the forward pass's 37.6 us at T = 250007, E = 160, and nothing backward.
template <int LPT, int U, int N>
__device__ __forceinline__ void softmax_rows(float (&z)[U][N], float2 (&mr)[U]) {
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float m = kNegInf;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, z[u][i]);
        m = group_max<LPT>(m);
        if (m == kNegInf) m = 0.0f;
        mr[u].x = m;
        s[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            z[u][i] = exp_from(z[u][i], m);
            s[u] += z[u][i];
        }
    }
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
#pragma unroll
    for (int u = 0; u < U; ++u) mr[u].y = s[u] > 0.0f ? __fdividef(1.0f, s[u]) : 0.0f;
}

// Rows that a group of lanes takes at a time, the next ones being loaded
// meanwhile: two of up to 8 values a lane.  One alone keeps 20 KB an SM in
// flight, and HBM wants about 35.
template <int N>
constexpr int rows_at_once = N <= 8 ? 2 : 1;

// ascending bounds inside [0, T]
__device__ bool bounds_ok(const int32_t *seq, int S, int T) {
    bool bad = false;
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        const int a = seq[s], b = seq[s + 1];
        if (a < 0 || b < a || b > T) bad = true;
    }
    return !__syncthreads_or(bad);
}

// The last s in [lo, S) with seq[s] <= t, where seq[lo] <= t: in steps that
// double, then halving.  A neighbour takes two loads, a far one 2 log2 of its
// distance; a walk through 65536 sequences took 14 ms of dependent loads.
__device__ __forceinline__ int sequence_at(const int32_t *seq, int S, int lo, int t) {
    int step = 1;
    while (lo + step < S && seq[lo + step] <= t) {
        lo += step;
        step *= 2;
    }
    int hi = min(S, lo + step) - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Workspace of the forward pass: chunk c of the tokens (`per` of them) meets
// sequence s in partial c + s, which no other pair has (both only ascend
// along the tokens), so a partial is written by one CTA and summed in order
// (terms added in a row: a lane's tokens of a chunk, T / 19456 with 8 lanes a
// token and T / 4864 with 32; then 8 warps, chunks / 32 partials and two trees):
//   psum [P, E] fp32, pcnt [P, E] int32, pn [P] int32,  P = chunks + S - 1.
// Pairs without a common token have no partial.
struct Joint {
    unsigned int done;    // combining CTAs that have left their shares
    int bad;              // the bounds are bad
};
template <int VEC, int LPT, int NC>
__global__ void __launch_bounds__(R_THREADS)
balance_partial_kernel(const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
                       const uint8_t *__restrict__ mask, const int32_t *__restrict__ seq, int S,
                       int T, int E, int k, int per, float *__restrict__ psum,
                       int32_t *__restrict__ pcnt, int32_t *__restrict__ pn, Joint *joint,
                       int32_t *dev_status) {
    using R = Row<VEC, LPT, NC>;
    constexpr int G = R_THREADS / LPT;        // token groups of the CTA
    constexpr int SPL = 32 / LPT;             // slots per lane
    constexpr int U = rows_at_once<R::N>;
    extern __shared__ float s_dyn[];          // [R_WARPS][E] sums, then [E] counts
    float *s_sum = s_dyn;
    int *s_cnt = reinterpret_cast<int *>(s_dyn + R_WARPS * E);
    __shared__ int s_n;
    const bool good = !seq || bounds_ok(seq, S, T);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        joint->done = 0;
        joint->bad = !good;
    }
    if (!good) return;                        // reported by the combining kernel
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = threadIdx.x % LPT, grp = threadIdx.x / LPT;
    const int c0 = blockIdx.x * per, c1 = min(T, c0 + per);
    const int end = seq ? min(c1, seq[S]) : c1;
    int s = 0;
    for (int a = seq ? max(c0, seq[0]) : c0, b; a < end; a = b) {
        if (seq) s = sequence_at(seq, S, s, a);
        b = seq ? min(c1, seq[s + 1]) : c1;
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += R_THREADS) s_cnt[e] = 0;
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        float acc[R::N];
#pragma unroll
        for (int i = 0; i < R::N; ++i) acc[i] = 0.0f;
        int n = 0;
        // the next tokens' rows and slots are loaded while these are summed
        float zn[U][R::N];
        int en[U][SPL];
        bool next_on[U];
        auto fetch = [&](int t0) {
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const int t = t0 + v * G + grp;
                next_on[v] = t < b && (!mask || mask[t] != 0);
#pragma unroll
                for (int i = 0; i < R::N; ++i) zn[v][i] = kNegInf;
#pragma unroll
                for (int u = 0; u < SPL; ++u) en[v][u] = 0;
                if (!next_on[v]) continue;
                R::load(logits + static_cast<int64_t>(t) * E, E, l, kNegInf, zn[v]);
#pragma unroll
                for (int u = 0; u < SPL; ++u)
                    if (u * LPT + l < k) en[v][u] = topk_idx[static_cast<int64_t>(t) * k + u * LPT + l];
            }
        };
        fetch(a);
        for (int t0 = a; t0 < b; t0 += U * G) {
            float z[U][R::N];
            int e[U][SPL];
            bool on[U];
#pragma unroll
            for (int v = 0; v < U; ++v) {
                on[v] = next_on[v];
#pragma unroll
                for (int i = 0; i < R::N; ++i) z[v][i] = zn[v][i];
#pragma unroll
                for (int u = 0; u < SPL; ++u) e[v][u] = en[v][u];
            }
            fetch(t0 + U * G);
            float2 mr[U];
            softmax_rows<LPT, U>(z, mr);
#pragma unroll
            for (int v = 0; v < U; ++v) {
#pragma unroll
                for (int i = 0; i < R::N; ++i) acc[i] = __fmaf_rn(z[v][i], mr[v].y, acc[i]);
                if (!on[v]) continue;
                n += l == 0;
#pragma unroll
                for (int u = 0; u < SPL; ++u) {
                    if (u * LPT + l >= k) continue;
                    if (e[v][u] >= 0 && e[v][u] < E)
                        atomicAdd(&s_cnt[e[v][u]], 1);
                    else
                        report(dev_status, MOE_DEV_BAD_EXPERT_ID);
                }
            }
        }
#pragma unroll
        for (int o = LPT; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < R::N; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (lane < LPT) {
#pragma unroll
            for (int i = 0; i < R::N; ++i) {
                const int e = R::col(l, i);
                if (e < E) s_sum[warp * E + e] = acc[i];
            }
        }
        if (n) atomicAdd(&s_n, n);
        __syncthreads();
        const int64_t p = static_cast<int64_t>(blockIdx.x) + s;
        for (int e = threadIdx.x; e < E; e += R_THREADS) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < R_WARPS; ++w) v += s_sum[w * E + e];
            psum[p * E + e] = v;
            pcnt[p * E + e] = s_cnt[e];
        }
        if (threadIdx.x == 0) pn[p] = s_n;
    }
}

// Joins the partials: a CTA takes C_COLS columns of one sequence, its 32 warps
// the chunks in turn, and leaves the columns' share of the loss; the CTA that
// finishes last adds the shares in order.  `joint` is written by the partial
// kernel's first CTA, which this kernel runs behind.
constexpr int C_COLS = 32;
constexpr int C_THREADS = 1024;

__global__ void __launch_bounds__(C_THREADS)
balance_combine_kernel(const float *__restrict__ psum, const int32_t *__restrict__ pcnt,
                       const int32_t *__restrict__ pn, const int32_t *__restrict__ seq, int S,
                       int T, int E, int k, int per, float coef, float *__restrict__ loss,
                       int32_t *__restrict__ counts, float *__restrict__ prob_mean,
                       int32_t *__restrict__ n_tokens, float *shares, Joint *joint,
                       int32_t *dev_status) {
    __shared__ float s_p[32][C_COLS + 1];
    __shared__ int s_c[32][C_COLS + 1];
    __shared__ int s_n[32];
    __shared__ bool s_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (joint->bad) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
            report(dev_status, MOE_DEV_BAD_OFFSETS);
        return;
    }
    const int s = blockIdx.x, e = blockIdx.y * C_COLS + lane;
    const int a = seq ? seq[s] : 0, b = seq ? seq[s + 1] : T;
    const int first = a / per, last = b > a ? (b - 1) / per : first - 1;
    float v = 0.0f;
    int cn = 0, n = 0;
    if (e < E) {
#pragma unroll 4
        for (int c = first + warp; c <= last; c += 32) {
            const int64_t at = (static_cast<int64_t>(c) + s) * E + e;
            v += psum[at];
            cn += pcnt[at];
        }
    }
    for (int c = first + static_cast<int>(threadIdx.x); c <= last; c += C_THREADS) n += pn[c + s];
    n = __reduce_add_sync(0xffffffffu, n);
    s_p[warp][lane] = v;
    s_c[warp][lane] = cn;
    if (lane == 0) s_n[warp] = n;
    __syncthreads();
    n = __reduce_add_sync(0xffffffffu, s_n[lane]);
    const float rn = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
    // warp w adds column w's 32 parts (its lanes in a tree)
    v = s_p[lane][warp];
    cn = __reduce_add_sync(0xffffffffu, s_c[lane][warp]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int col = blockIdx.y * C_COLS + warp;
    const float pm = v * rn;
    __syncthreads();
    if (lane == 0) {
        s_p[0][warp] = col < E ? static_cast<float>(cn) * pm : 0.0f;
        if (col < E) {
            prob_mean[static_cast<int64_t>(s) * E + col] = pm;
            counts[static_cast<int64_t>(s) * E + col] = cn;
        }
    }
    __syncthreads();
    if (warp == 0) {
        float share = s_p[0][lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) share += __shfl_xor_sync(0xffffffffu, share, o);
        if (lane == 0) {
            shares[static_cast<int64_t>(s) * gridDim.y + blockIdx.y] = share * rn;
            if (blockIdx.y == 0) n_tokens[s] = n;
            __threadfence();
            s_last = atomicAdd(&joint->done, 1u) == gridDim.x * gridDim.y - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // the last CTA: every thread its strided shares in order, then a tree
    const int total = static_cast<int>(gridDim.x * gridDim.y);
    float sum = 0.0f;
    int live = 0;
    for (int i = threadIdx.x; i < total; i += C_THREADS) sum += __ldcg(shares + i);
    for (int i = threadIdx.x; i < S; i += C_THREADS) live += __ldcg(n_tokens + i) > 0;
    live = __reduce_add_sync(0xffffffffu, live);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
        s_p[1][warp] = sum;
        s_n[warp] = live;
    }
    __syncthreads();
    if (warp == 0) {
        sum = s_p[1][lane];
        live = __reduce_add_sync(0xffffffffu, s_n[lane]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0)
            *loss = live > 0
                        ? coef * static_cast<float>(E) / (static_cast<float>(k) * live) * sum
                        : 0.0f;
    }
}

// The gradient: a group of LPT lanes per token; slot j belongs to lane
// j % LPT, which reads its own logit again (in L1) for the slot's probability.
template <int VEC, int LPT, int NC>
__global__ void __launch_bounds__(R_THREADS)
topk_backward_kernel(const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
                     const float *__restrict__ d_topk_w, const uint8_t *__restrict__ mask,
                     const int32_t *__restrict__ seq, int S, const int32_t *__restrict__ counts,
                     const int32_t *__restrict__ n_tokens, const float *__restrict__ d_loss,
                     float coef, int T, int E, int k, bool renorm, int per,
                     float *__restrict__ d_logits, int32_t *dev_status) {
    using R = Row<VEC, LPT, NC>;
    constexpr int G = R_THREADS / LPT;
    constexpr int SPL = 32 / LPT;              // slots per lane
    constexpr int U = rows_at_once<R::N>;
    __shared__ int s_live;
    const int l = threadIdx.x % LPT, grp = threadIdx.x / LPT;
    extern __shared__ float4 s_buf[];          // [G][columns]: a group's slot terms
    float *buf = reinterpret_cast<float *>(s_buf) + grp * (LPT * R::N);
    if (d_topk_w)
        for (int i = l; i < LPT * R::N; i += LPT) buf[i] = 0.0f;
    float unit = 0.0f;                         // coef E d_loss / (S+ k)
    if (counts) {
        if (seq && !bounds_ok(seq, S, T)) {
            if (blockIdx.x == 0 && threadIdx.x == 0) report(dev_status, MOE_DEV_BAD_OFFSETS);
            return;
        }
        if (threadIdx.x == 0) s_live = 0;
        __syncthreads();
        int live = 0;
        for (int s = threadIdx.x; s < S; s += R_THREADS) live += n_tokens[s] > 0;
        if (live) atomicAdd(&s_live, live);
        __syncthreads();
        if (s_live > 0)
            unit = coef * static_cast<float>(E) / (static_cast<float>(k) * s_live) *
                   (d_loss ? *d_loss : 1.0f);
    }
    // last chunk first: the forward pass left the ends of the logits in L2
    const int c0 = (gridDim.x - 1 - blockIdx.x) * per, c1 = min(T, c0 + per);
    int seq_end = -1;                          // the held sequence's end
    int s_cur = 0;
    bool inside = false;
    float cnt[R::N];
    float scale = 0.0f;
#pragma unroll
    for (int i = 0; i < R::N; ++i) cnt[i] = 0.0f;
    // the next tokens' rows, slots and weights' gradients are loaded meanwhile
    float zn[U][R::N], dn[U][SPL];
    int en[U][SPL];
    bool next_on[U];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const int t = t0 + v * G + grp;
            next_on[v] = t < c1 && (!mask || mask[t] != 0);
#pragma unroll
            for (int i = 0; i < R::N; ++i) zn[v][i] = kNegInf;
#pragma unroll
            for (int u = 0; u < SPL; ++u) {
                en[v][u] = -1;
                dn[v][u] = 0.0f;
            }
            if (!next_on[v]) continue;
            R::load(logits + static_cast<int64_t>(t) * E, E, l, kNegInf, zn[v]);
            if (!d_topk_w) continue;
#pragma unroll
            for (int u = 0; u < SPL; ++u)
                if (u * LPT + l < k) {
                    en[v][u] = topk_idx[static_cast<int64_t>(t) * k + u * LPT + l];
                    dn[v][u] = d_topk_w[static_cast<int64_t>(t) * k + u * LPT + l];
                }
        }
    };
    fetch(c0);
    for (int t0 = c0; t0 < c1; t0 += U * G) {
        float p[U][R::N], g[U][SPL], z[U][SPL];
        int idx[U][SPL];
        bool on[U];
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const int t = t0 + v * G + grp;
            on[v] = next_on[v];
#pragma unroll
            for (int i = 0; i < R::N; ++i) p[v][i] = zn[v][i];
#pragma unroll
            for (int u = 0; u < SPL; ++u) {
                idx[v][u] = en[v][u];
                g[v][u] = dn[v][u];
                z[v][u] = kNegInf;
                if (!d_topk_w || !on[v] || u * LPT + l >= k) continue;
                if (idx[v][u] >= 0 && idx[v][u] < E) {
                    z[v][u] = __ldg(logits + static_cast<int64_t>(t) * E + idx[v][u]);
                } else {
                    report(dev_status, MOE_DEV_BAD_EXPERT_ID);
                    idx[v][u] = -1;
                    g[v][u] = 0.0f;
                }
            }
        }
        fetch(t0 + U * G);
        float2 mr[U];
        softmax_rows<LPT, U>(p, mr);
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const int t = t0 + v * G + grp;
            if (counts && on[v] && t >= seq_end) {
                // the token's sequence, its counts and its factor
                int s = s_cur;
                if (seq && t < seq[0]) {
                    seq_end = seq[0];
                } else if (seq) {
                    s = sequence_at(seq, S, s_cur, t);
                    inside = t < seq[s + 1];
                    seq_end = inside ? seq[s + 1] : 0x7fffffff;
                } else {
                    inside = true;
                    seq_end = 0x7fffffff;
                }
                s_cur = s;
                scale = 0.0f;
                if (inside) {
                    const float n = static_cast<float>(max(n_tokens[s], 1));
                    scale = unit / (n * n);
#pragma unroll
                    for (int i = 0; i < R::N; ++i) {
                        const int e = R::col(l, i);
                        cnt[i] = e < E ? static_cast<float>(counts[static_cast<int64_t>(s) * E + e])
                                       : 0.0f;
                    }
                }
            }
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < R::N; ++i) dot = __fmaf_rn(p[v][i], cnt[i], dot);
            dot = group_sum<LPT>(dot) * mr[v].y;
            float sub = 0.0f;                  // sum_l p_l dw_l without renormalisation
            if (d_topk_w) {
                float w[SPL], ws = 0.0f, wd = 0.0f, m = mr[v].x;
                if (renorm) {
                    m = kNegInf;
#pragma unroll
                    for (int u = 0; u < SPL; ++u) m = fmaxf(m, z[v][u]);
                    m = group_max<LPT>(m);
                    if (m == kNegInf) m = 0.0f;
                }
#pragma unroll
                for (int u = 0; u < SPL; ++u) {
                    w[u] = exp_from(z[v][u], m);
                    if (!renorm) w[u] *= mr[v].y;
                    ws += w[u];
                    wd += w[u] * g[v][u];
                }
                wd = group_sum<LPT>(wd);
                if (renorm) {
                    ws = group_sum<LPT>(ws);
                    const float r = ws > 0.0f ? __fdividef(1.0f, ws) : 0.0f;
                    wd *= r;
#pragma unroll
                    for (int u = 0; u < SPL; ++u) g[v][u] = w[u] * r * (g[v][u] - wd);
                } else {
                    sub = wd;
#pragma unroll
                    for (int u = 0; u < SPL; ++u) g[v][u] *= w[u];
                }
            }
            // p (scale (c - dot) - sub), p = e * mr.y
            const float rs = scale * mr[v].y, rsub = sub * mr[v].y;
#pragma unroll
            for (int i = 0; i < R::N; ++i) p[v][i] *= __fmaf_rn(rs, cnt[i] - dot, -rsub);
            if (d_topk_w) {
                // Each slot's term goes to the lane of its column through the
                // group's row of shared memory (zeros between tokens).  A slot
                // whose mark another one has overwritten names the same expert.
                __syncwarp();
#pragma unroll
                for (int u = 0; u < SPL; ++u)
                    if (idx[v][u] >= 0) buf[idx[v][u]] = __int_as_float(1 + u * LPT + l);
                __syncwarp();
                bool twice = false;
#pragma unroll
                for (int u = 0; u < SPL; ++u)
                    if (idx[v][u] >= 0) twice |= __float_as_int(buf[idx[v][u]]) != 1 + u * LPT + l;
                twice = __any_sync(0xffffffffu, twice);
                __syncwarp();
#pragma unroll
                for (int u = 0; u < SPL; ++u)
                    if (idx[v][u] >= 0) buf[idx[v][u]] = twice ? 0.0f : g[v][u];
                if (twice) {                   // in slot order
                    for (int j = 0; j < k; ++j) {
                        __syncwarp();
#pragma unroll
                        for (int u = 0; u < SPL; ++u)
                            if (j == u * LPT + l && idx[v][u] >= 0) buf[idx[v][u]] += g[v][u];
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < R::N; ++i) p[v][i] += buf[R::col(l, i)];
                __syncwarp();
#pragma unroll
                for (int u = 0; u < SPL; ++u)
                    if (idx[v][u] >= 0) buf[idx[v][u]] = 0.0f;
            }
            if (t < c1) {
                if (!on[v]) {
#pragma unroll
                    for (int i = 0; i < R::N; ++i) p[v][i] = 0.0f;
                }
                R::store(d_logits + static_cast<int64_t>(t) * E, E, l, p[v]);
            }
        }
    }
}

// finalize's backward: for slot j of token t with row r
//   d_y[r] = topk_w[t, j] * d_out[t],  d_topk_w[t, j] = <d_out[t], y[r]>.
// A CTA takes U slots of one token: d_out is read once for them and held in
// registers vector by vector; HBM bound (the rows in, their gradients out):
// 16384 x 4096, 8 slots, bf16: 345 us, 6.6 TB/s of 2.28 GB.
template <int U, bool Y_F32, bool D_F32>
__global__ void __launch_bounds__(R_THREADS)
finalize_backward_kernel(const void *__restrict__ d_out, const void *__restrict__ y_exp,
                         const int32_t *__restrict__ row_idx, const float *__restrict__ topk_w,
                         int T, int H, int k, int n, void *__restrict__ d_y,
                         float *__restrict__ d_w, int32_t *dev_status) {
    __shared__ float s_part[R_WARPS][U];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nvec = H / 8;
    const int parts = (k + U - 1) / U;
    const int64_t units = static_cast<int64_t>(T) * parts;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int t = static_cast<int>(unit / parts);
        const int j0 = static_cast<int>(unit % parts) * U;
        int row[U];
        float w[U], acc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u;
            const int64_t at = static_cast<int64_t>(t) * k + j;
            row[u] = j < k ? __ldg(row_idx + at) : -1;
            w[u] = j < k ? __ldg(topk_w + at) : 0.0f;
            if (row[u] >= n) {
                if (threadIdx.x == 0) report(dev_status, MOE_DEV_BAD_OFFSETS);
                row[u] = -1;
            }
            acc[u] = 0.0f;
        }
        for (int v = threadIdx.x; v < nvec; v += R_THREADS) {
            float d[8];
            if (D_F32) {
                const float4 *src = reinterpret_cast<const float4 *>(
                                        static_cast<const float *>(d_out) +
                                        static_cast<int64_t>(t) * H) + 2 * v;
                const float4 a = __ldg(src), b = __ldg(src + 1);
                d[0] = a.x; d[1] = a.y; d[2] = a.z; d[3] = a.w;
                d[4] = b.x; d[5] = b.y; d[6] = b.z; d[7] = b.w;
            } else {
                const uint4 a = __ldg(reinterpret_cast<const uint4 *>(
                                          static_cast<const uint16_t *>(d_out) +
                                          static_cast<int64_t>(t) * H) + v);
                const uint32_t wd[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d[2 * i] = __uint_as_float(wd[i] << 16);
                    d[2 * i + 1] = __uint_as_float(wd[i] & 0xFFFF0000u);
                }
            }
            if (Y_F32) {
                float4 qa[U], qb[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (row[u] >= 0) {
                        const float4 *src = reinterpret_cast<const float4 *>(
                                                static_cast<const float *>(y_exp) +
                                                static_cast<int64_t>(row[u]) * H) + 2 * v;
                        qa[u] = __ldg(src);
                        qb[u] = __ldg(src + 1);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (row[u] >= 0) {
                        acc[u] += d[0] * qa[u].x + d[1] * qa[u].y + d[2] * qa[u].z + d[3] * qa[u].w +
                                  d[4] * qb[u].x + d[5] * qb[u].y + d[6] * qb[u].z + d[7] * qb[u].w;
                        float4 *dst = reinterpret_cast<float4 *>(
                                          static_cast<float *>(d_y) +
                                          static_cast<int64_t>(row[u]) * H) + 2 * v;
                        dst[0] = make_float4(w[u] * d[0], w[u] * d[1], w[u] * d[2], w[u] * d[3]);
                        dst[1] = make_float4(w[u] * d[4], w[u] * d[5], w[u] * d[6], w[u] * d[7]);
                    }
            } else {
                uint4 q[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (row[u] >= 0)
                        q[u] = __ldg(reinterpret_cast<const uint4 *>(
                                         static_cast<const uint16_t *>(y_exp) +
                                         static_cast<int64_t>(row[u]) * H) + v);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (row[u] >= 0) {
                        const uint32_t wd[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            acc[u] += d[2 * i] * __uint_as_float(wd[i] << 16);
                            acc[u] += d[2 * i + 1] * __uint_as_float(wd[i] & 0xFFFF0000u);
                            o[i] = bf16x2(w[u] * d[2 * i], w[u] * d[2 * i + 1]);
                        }
                        *(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(d_y) +
                                                    static_cast<int64_t>(row[u]) * H) + v) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
            }
        }
        __syncthreads();                       // the previous unit's sums are read
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s = acc[u];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) s_part[warp][u] = s;
        }
        __syncthreads();
        if (threadIdx.x < U && j0 + threadIdx.x < k) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < R_WARPS; ++i) s += s_part[i][threadIdx.x];
            d_w[static_cast<int64_t>(t) * k + j0 + threadIdx.x] = s;
        }
    }
}

inline bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Chunks and their tokens: `per_sm` CTAs per SM, at least 32 tokens each.  The
// forward pass takes the four that are resident at once, since its chunks'
// partial sums are joined afterwards; the backward pass three times as many,
// so that the last round of its three or four resident ones is short.
struct Chunks {
    int count, per;
};
Chunks chunks_of(int T, int per_sm = 4) {
    const int64_t most = static_cast<int64_t>(num_sms()) * per_sm;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(most, ceil_div(T, 32)));
    const int per = static_cast<int>(std::max<int64_t>(1, ceil_div(T, want)));
    return {static_cast<int>(std::max<int64_t>(1, ceil_div(T, per))), per};
}

// Calls f(Row shape) with the smallest shape that holds E columns; whole
// float4s need 16-byte aligned rows.
template <typename F>
void with_row_shape(int E, bool vec, F f) {
#define MOE_SHAPE(V, L, N) f(std::integral_constant<int, V>(), std::integral_constant<int, L>(), std::integral_constant<int, N>())
    if (vec) {
        if (E <= 32) MOE_SHAPE(4, 8, 1);
        else if (E <= 64) MOE_SHAPE(4, 8, 2);
        else if (E <= 128) MOE_SHAPE(4, 8, 4);
        else if (E <= 192) MOE_SHAPE(4, 16, 3);
        else if (E <= 256) MOE_SHAPE(4, 16, 4);
        else if (E <= 384) MOE_SHAPE(4, 32, 3);
        else if (E <= 512) MOE_SHAPE(4, 32, 4);
        else MOE_SHAPE(4, 32, 8);
    } else {
        if (E <= 32) MOE_SHAPE(1, 32, 1);
        else if (E <= 64) MOE_SHAPE(1, 32, 2);
        else if (E <= 128) MOE_SHAPE(1, 32, 4);
        else if (E <= 256) MOE_SHAPE(1, 32, 8);
        else if (E <= 512) MOE_SHAPE(1, 32, 16);
        else MOE_SHAPE(1, 32, 32);
    }
#undef MOE_SHAPE
}

bool whole_vectors(int E, const void *a, const void *b) {
    return E % 4 == 0 && a16(a) && (!b || a16(b));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_balance_loss_workspace_size(int32_t T, int32_t E, int32_t S,
                                                        size_t *bytes) {
    if (!bytes || T < 0 || E <= 0 || S <= 0) return MOE_ERR_INVALID_ARG;
    if (E > 1024 || S > 65536 || T > (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
    const size_t P = static_cast<size_t>(chunks_of(T).count) + S;
    // the partials, the shares of the loss and what joins them
    *bytes = 2 * align256(P * E * 4) + align256(P * 4) +
             align256(static_cast<size_t>(S) * ceil_div(E, C_COLS) * 4) + 256;
    return MOE_OK;
}

extern "C" moe_status_t moe_balance_loss(const float *logits, const int32_t *topk_idx,
                                         const uint8_t *token_mask, const int32_t *seq_offsets,
                                         int32_t S, int32_t T, int32_t E, int32_t k, float coef,
                                         float *loss, int32_t *counts, float *prob_mean,
                                         int32_t *n_tokens, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status,
                                         moe_stream_t stream) {
    if (T < 0 || E <= 0 || k <= 0 || S <= 0 || (!seq_offsets && S != 1)) return MOE_ERR_INVALID_ARG;
    if (E > 1024 || k > 32 || k > E) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(T) * k >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    size_t need = 0;
    const moe_status_t st = moe_balance_loss_workspace_size(T, E, S, &need);
    if (st != MOE_OK) return st;
    if (!loss || !counts || !prob_mean || !n_tokens || (T > 0 && (!logits || !topk_idx)))
        return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Chunks ch = chunks_of(T);
    const size_t P = static_cast<size_t>(ch.count) + S;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *psum = reinterpret_cast<float *>(ws);
    int32_t *pcnt = reinterpret_cast<int32_t *>(ws + align256(P * E * 4));
    int32_t *pn = reinterpret_cast<int32_t *>(ws + 2 * align256(P * E * 4));
    float *shares = reinterpret_cast<float *>(ws + 2 * align256(P * E * 4) + align256(P * 4));
    Joint *joint = reinterpret_cast<Joint *>(ws + need - 256);
    if (T == 0) {
        const size_t SE = static_cast<size_t>(S) * E * 4;
        if (cudaMemsetAsync(loss, 0, 4, s) != cudaSuccess ||
            cudaMemsetAsync(counts, 0, SE, s) != cudaSuccess ||
            cudaMemsetAsync(prob_mean, 0, SE, s) != cudaSuccess ||
            cudaMemsetAsync(n_tokens, 0, static_cast<size_t>(S) * 4, s) != cudaSuccess)
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    const size_t smem = static_cast<size_t>(R_WARPS + 1) * E * 4;   // at most 36 KB
    with_row_shape(E, whole_vectors(E, logits, nullptr), [&](auto v, auto l, auto n) {
        balance_partial_kernel<v.value, l.value, n.value><<<ch.count, R_THREADS, smem, s>>>(
            logits, topk_idx, token_mask, seq_offsets, S, T, E, k, ch.per, psum, pcnt, pn, joint,
            dev_status);
    });
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(S), static_cast<unsigned>(ceil_div(E, C_COLS)));
    balance_combine_kernel<<<grid, C_THREADS, 0, s>>>(psum, pcnt, pn, seq_offsets, S, T, E, k,
                                                      ch.per, coef, loss, counts, prob_mean,
                                                      n_tokens, shares, joint, dev_status);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status_t moe_gate_topk_backward(
    const float *logits, const int32_t *topk_idx, const float *d_topk_w, const uint8_t *token_mask,
    const int32_t *seq_offsets, int32_t S, const int32_t *counts, const int32_t *n_tokens,
    const float *d_loss, float coef, int32_t T, int32_t E, int32_t k, uint32_t flags,
    float *d_logits, int32_t *dev_status, moe_stream_t stream) {
    if (T < 0 || E <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (E > 1024 || k > 32 || k > E || T > (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(T) * k >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!counts != !n_tokens) return MOE_ERR_INVALID_ARG;
    if (counts && (S <= 0 || (!seq_offsets && S != 1))) return MOE_ERR_INVALID_ARG;
    if (counts && S > 65536) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || !d_logits || (d_topk_w && !topk_idx)) return MOE_ERR_INVALID_ARG;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Chunks ch = chunks_of(T, 12);
    with_row_shape(E, whole_vectors(E, logits, d_logits), [&](auto v, auto l, auto n) {
        // a row of columns per group: at most 32 KB
        const size_t smem = static_cast<size_t>(R_THREADS) * v.value * n.value * 4;
        topk_backward_kernel<v.value, l.value, n.value><<<ch.count, R_THREADS, smem, s>>>(
            logits, topk_idx, d_topk_w, token_mask, seq_offsets, S, counts, n_tokens, d_loss, coef,
            T, E, k, (flags & MOE_RENORM) != 0, ch.per, d_logits, dev_status);
    });
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status_t moe_finalize_routing_backward(const void *d_out, const void *y_exp,
                                                      const int32_t *expanded_row_idx,
                                                      const float *topk_w, int32_t T, int32_t H,
                                                      int32_t k, uint32_t flags, void *d_y_exp,
                                                      float *d_topk_w, int32_t *dev_status,
                                                      moe_stream_t stream) {
    if (T < 0 || H <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (H % 8 != 0 || k > 32) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(T) * k >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!d_out || !y_exp || !expanded_row_idx || !topk_w || !d_y_exp || !d_topk_w)
        return MOE_ERR_INVALID_ARG;
    if (!a16(d_out) || !a16(y_exp) || !a16(d_y_exp)) return MOE_ERR_INVALID_ARG;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool yf = (flags & MOE_Y_F32) != 0, df = (flags & MOE_OUT_F32) != 0;
    // few tokens: a CTA per slot, so that the rows spread over the SMs
    const bool few = static_cast<int64_t>(T) < 2 * num_sms();
    const int64_t units = few ? static_cast<int64_t>(T) * k : static_cast<int64_t>(T) * ceil_div(k, 8);
    const int grid = static_cast<int>(std::min<int64_t>(units, static_cast<int64_t>(num_sms()) * 64));
#define MOE_FB(U, YF, DF)                                                                     \
    finalize_backward_kernel<U, YF, DF><<<grid, R_THREADS, 0, s>>>(                           \
        d_out, y_exp, expanded_row_idx, topk_w, T, H, k, T * k, d_y_exp, d_topk_w, dev_status)
    if (few) {
        if (yf && df) MOE_FB(1, true, true);
        else if (yf) MOE_FB(1, true, false);
        else if (df) MOE_FB(1, false, true);
        else MOE_FB(1, false, false);
    } else {
        if (yf && df) MOE_FB(8, true, true);
        else if (yf) MOE_FB(8, true, false);
        else if (df) MOE_FB(8, false, true);
        else MOE_FB(8, false, false);
    }
#undef MOE_FB
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
