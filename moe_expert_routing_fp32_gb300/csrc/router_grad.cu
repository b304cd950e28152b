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
// Bound: the logits are read once by each pass and the gradient written once.
// A group of lanes (16 for E <= 64 in whole float4s, else 32) holds one
// token's row in registers; nothing is staged through shared memory.
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
                *reinterpret_cast<float4 *>(row + e) =
                    make_float4(z[c * 4], z[c * 4 + 1], z[c * 4 + 2], z[c * 4 + 3]);
            else
                row[e] = z[c];
        }
    }
};

template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// z -> p in place; returns (max, 1 / sum).  A row with no finite logit gives
// zeros.
template <int LPT, int N>
__device__ __forceinline__ float2 softmax_row(float (&z)[N]) {
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, z[i]);
    m = group_max<LPT>(m);
    if (m == kNegInf) m = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        z[i] = expf(z[i] - m);
        s += z[i];
    }
    s = group_sum<LPT>(s);
    const float r = s > 0.0f ? 1.0f / s : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] *= r;
    return make_float2(m, r);
}

// ascending bounds inside [0, T]
__device__ bool bounds_ok(const int32_t *seq, int S, int T) {
    bool bad = false;
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        const int a = seq[s], b = seq[s + 1];
        if (a < 0 || b < a || b > T) bad = true;
    }
    return !__syncthreads_or(bad);
}

// Workspace of the forward pass: chunk c of the tokens (`per` of them) meets
// sequence s in partial c + s, which no other pair has (both only ascend
// along the tokens), so a partial is written by one CTA and summed in order:
//   psum [P, E] fp32, pcnt [P, E] int32, pn [P] int32,  P = chunks + S - 1.
template <int VEC, int LPT, int NC>
__global__ void __launch_bounds__(R_THREADS)
balance_partial_kernel(const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
                       const uint8_t *__restrict__ mask, const int32_t *__restrict__ seq, int S,
                       int T, int E, int k, int per, float *__restrict__ psum,
                       int32_t *__restrict__ pcnt, int32_t *__restrict__ pn, int32_t *dev_status) {
    using R = Row<VEC, LPT, NC>;
    constexpr int G = R_THREADS / LPT;        // token groups of the CTA
    extern __shared__ float s_dyn[];          // [R_WARPS][E] sums, then [E] counts
    float *s_sum = s_dyn;
    int *s_cnt = reinterpret_cast<int *>(s_dyn + R_WARPS * E);
    __shared__ int s_n;
    if (seq && !bounds_ok(seq, S, T)) return;   // reported by the combining kernel
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = threadIdx.x % LPT, grp = threadIdx.x / LPT;
    const int c0 = blockIdx.x * per, c1 = min(T, c0 + per);
    int s = 0;
    if (seq) {
        int hi = S - 1;                        // last sequence that starts at or before c0
        while (s < hi) {
            const int mid = (s + hi + 1) >> 1;
            if (seq[mid] <= c0)
                s = mid;
            else
                hi = mid - 1;
        }
    }
    for (; s < S; ++s) {
        const int a = seq ? max(c0, seq[s]) : c0, b = seq ? min(c1, seq[s + 1]) : c1;
        if (seq && seq[s] >= c1 && s > 0) break;
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += R_THREADS) s_cnt[e] = 0;
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        float acc[R::N];
#pragma unroll
        for (int i = 0; i < R::N; ++i) acc[i] = 0.0f;
        int n = 0;
        for (int t0 = a; t0 < b; t0 += G) {
            const int t = t0 + grp;
            const bool on = t < b && (!mask || mask[t] != 0);
            float z[R::N];
#pragma unroll
            for (int i = 0; i < R::N; ++i) z[i] = kNegInf;
            if (on) R::load(logits + static_cast<int64_t>(t) * E, E, l, kNegInf, z);
            softmax_row<LPT>(z);
#pragma unroll
            for (int i = 0; i < R::N; ++i) acc[i] += z[i];
            if (on) {
                n += l == 0;
                for (int j = l; j < k; j += LPT) {
                    const int e = topk_idx[static_cast<int64_t>(t) * k + j];
                    if (e >= 0 && e < E)
                        atomicAdd(&s_cnt[e], 1);
                    else
                        report(dev_status, MOE_DEV_BAD_EXPERT_ID);
                }
            }
        }
        if (LPT == 16) {
#pragma unroll
            for (int i = 0; i < R::N; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 16);
        }
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

// One cluster of C_CTAS joins the partials: CTA r takes the columns
// [r E / C, (r + 1) E / C) of every sequence, in chunk order, and its share of
// the loss; the shares meet in CTA 0.
constexpr int C_CTAS = 8;

__global__ void __cluster_dims__(C_CTAS, 1, 1) __launch_bounds__(R_THREADS)
balance_combine_kernel(const float *__restrict__ psum, const int32_t *__restrict__ pcnt,
                       const int32_t *__restrict__ pn, const int32_t *__restrict__ seq, int S,
                       int T, int E, int k, int per, float coef, float *__restrict__ loss,
                       int32_t *__restrict__ counts, float *__restrict__ prob_mean,
                       int32_t *__restrict__ n_tokens, int32_t *dev_status) {
    __shared__ float s_share[C_CTAS];
    __shared__ float s_red[R_WARPS];
    __shared__ float s_p[R_THREADS];
    __shared__ int s_c[R_THREADS];
    __shared__ int s_nred[R_WARPS];
    const uint32_t rank = cluster_ctarank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool ok = !seq || bounds_ok(seq, S, T);
    if (!ok && rank == 0 && tid == 0) report(dev_status, MOE_DEV_BAD_OFFSETS);
    const int e0 = static_cast<int>(static_cast<int64_t>(rank) * E / C_CTAS);
    const int e1 = static_cast<int>(static_cast<int64_t>(rank + 1) * E / C_CTAS);
    const int cols = e1 - e0;
    int width = 1;                             // columns side by side: a power of two
    while (width < cols && width < 32) width <<= 1;
    const int par = R_THREADS / width;         // chunks side by side
    float share = 0.0f;
    int live = 0;
    for (int s = 0; ok && s < S; ++s) {
        const int a = seq ? seq[s] : 0, b = seq ? seq[s + 1] : T;
        const int f = a / per, last = b > a ? (b - 1) / per : f - 1;
        int n = 0;
        for (int c = f + tid; c <= last; c += R_THREADS) n += pn[c + s];
        n = __reduce_add_sync(0xffffffffu, n);
        __syncthreads();
        if (lane == 0) s_nred[warp] = n;
        __syncthreads();
        n = 0;
#pragma unroll
        for (int w = 0; w < R_WARPS; ++w) n += s_nred[w];
        if (rank == 0 && tid == 0) n_tokens[s] = n;
        live += n > 0;
        const float rn = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
        const int used = min(par, last - f + 1);
        float dot = 0.0f;
        for (int eb = e0; eb < e1; eb += width) {
            const int e = eb + tid % width;
            float v = 0.0f;
            int cn = 0;
            if (e < e1) {
                for (int c = f + tid / width; c <= last; c += par) {
                    const int64_t at = (static_cast<int64_t>(c) + s) * E + e;
                    v += psum[at];
                    cn += pcnt[at];
                }
            }
            __syncthreads();
            s_p[tid] = v;
            s_c[tid] = cn;
            __syncthreads();
            if (tid < width && e < e1) {
                v = 0.0f;
                cn = 0;
                for (int c = 0; c < used; ++c) {
                    v += s_p[c * width + tid];
                    cn += s_c[c * width + tid];
                }
                const float pm = v * rn;
                prob_mean[static_cast<int64_t>(s) * E + e] = pm;
                counts[static_cast<int64_t>(s) * E + e] = cn;
                dot += static_cast<float>(cn) * pm;
            }
        }
        share += dot * rn;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) share += __shfl_xor_sync(0xffffffffu, share, o);
    if (lane == 0) s_red[warp] = share;
    __syncthreads();
    cluster_sync_all();                        // every CTA of the cluster has started
    if (tid == 0) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < R_WARPS; ++w) v += s_red[w];
        st_shared_cluster_u32(mapa_shared(smem_u32(&s_share[rank]), 0), __float_as_uint(v));
    }
    cluster_sync_all();
    if (rank == 0 && tid == 0 && ok) {
        float v = 0.0f;
#pragma unroll
        for (int r = 0; r < C_CTAS; ++r) v += s_share[r];
        *loss = live > 0 ? coef * static_cast<float>(E) / (static_cast<float>(k) * live) * v : 0.0f;
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
    __shared__ int s_live;
    const int l = threadIdx.x % LPT, grp = threadIdx.x / LPT;
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
    const int c0 = blockIdx.x * per, c1 = min(T, c0 + per);
    int seq_end = -1;                          // the held sequence's end
    int s_cur = 0;
    bool inside = false;
    float cnt[R::N];
    float scale = 0.0f;
#pragma unroll
    for (int i = 0; i < R::N; ++i) cnt[i] = 0.0f;
    for (int t0 = c0; t0 < c1; t0 += G) {
        const int t = t0 + grp;
        const bool on = t < c1 && (!mask || mask[t] != 0);
        if (counts && on && t >= seq_end) {
            // the token's sequence, its counts and its factor
            int s = s_cur;
            if (seq) {
                while (s < S && seq[s + 1] <= t) ++s;
                inside = s < S && seq[s] <= t;
                seq_end = s < S ? (inside ? seq[s + 1] : seq[s]) : 0x7fffffff;
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
        const float *row = logits + static_cast<int64_t>(t) * E;
        float p[R::N];
#pragma unroll
        for (int i = 0; i < R::N; ++i) p[i] = kNegInf;
        if (on) R::load(row, E, l, kNegInf, p);
        const float2 mr = softmax_row<LPT>(p);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < R::N; ++i) dot += p[i] * cnt[i];
        dot = group_sum<LPT>(dot);
        float sub = 0.0f;                      // sum_l p_l dw_l without renormalisation
        int idx[SPL];
        float g[SPL];
        if (d_topk_w) {
            float z[SPL], m = kNegInf;
#pragma unroll
            for (int u = 0; u < SPL; ++u) {
                const int j = u * LPT + l;
                idx[u] = -1;
                g[u] = 0.0f;
                z[u] = kNegInf;
                if (on && j < k) {
                    const int e = topk_idx[static_cast<int64_t>(t) * k + j];
                    if (e >= 0 && e < E) {
                        idx[u] = e;
                        g[u] = d_topk_w[static_cast<int64_t>(t) * k + j];
                        z[u] = __ldg(row + e);
                    } else {
                        report(dev_status, MOE_DEV_BAD_EXPERT_ID);
                    }
                }
                m = fmaxf(m, z[u]);
            }
            float w[SPL], ws = 0.0f, wd = 0.0f;
            if (renorm) {
                m = group_max<LPT>(m);
                if (m == kNegInf) m = 0.0f;
            } else {
                m = mr.x;
            }
#pragma unroll
            for (int u = 0; u < SPL; ++u) {
                w[u] = expf(z[u] - m);
                if (!renorm) w[u] *= mr.y;
                ws += w[u];
                wd += w[u] * g[u];
            }
            wd = group_sum<LPT>(wd);
            if (renorm) {
                ws = group_sum<LPT>(ws);
                const float r = ws > 0.0f ? 1.0f / ws : 0.0f;
                wd *= r;
#pragma unroll
                for (int u = 0; u < SPL; ++u) g[u] = w[u] * r * (g[u] - wd);
            } else {
                sub = wd;
#pragma unroll
                for (int u = 0; u < SPL; ++u) g[u] *= w[u];
            }
        }
#pragma unroll
        for (int i = 0; i < R::N; ++i) p[i] *= scale * (cnt[i] - dot) - sub;
        if (d_topk_w) {
            // hand every slot's term to the lane that holds its column, in slot order
#pragma unroll
            for (int u = 0; u < SPL; ++u) {
                const int slots = min(LPT, k - u * LPT);
                for (int j = 0; j < slots; ++j) {
                    const int e = __shfl_sync(0xffffffffu, idx[u], j, LPT);
                    const float v = __shfl_sync(0xffffffffu, g[u], j, LPT);
#pragma unroll
                    for (int i = 0; i < R::N; ++i)
                        if (R::col(l, i) == e) p[i] += v;
                }
            }
        }
        if (t < c1) {
            if (!on) {
#pragma unroll
                for (int i = 0; i < R::N; ++i) p[i] = 0.0f;
            }
            R::store(d_logits + static_cast<int64_t>(t) * E, E, l, p);
        }
    }
}

// finalize's backward: for slot j of token t with row r
//   d_y[r] = topk_w[t, j] * d_out[t],  d_topk_w[t, j] = <d_out[t], y[r]>.
// A CTA takes U slots of one token: d_out is read once for them and held in
// registers vector by vector; HBM bound (the rows in, their gradients out).
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

// Chunks of the forward pass and their tokens: about four CTAs per SM, at
// least 32 tokens each (two passes of a CTA's sixteen groups).
struct Chunks {
    int count, per;
};
Chunks chunks_of(int T) {
    const int64_t most = static_cast<int64_t>(num_sms()) * 4;
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
        if (E <= 64) MOE_SHAPE(4, 16, 1);
        else if (E <= 128) MOE_SHAPE(4, 32, 1);
        else if (E <= 256) MOE_SHAPE(4, 32, 2);
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
    if (E > 1024 || S > 65536) return MOE_ERR_UNSUPPORTED_SHAPE;
    const size_t P = static_cast<size_t>(chunks_of(T).count) + S;
    *bytes = 2 * align256(P * E * 4) + align256(P * 4);
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
    if (T > 0) {
        const size_t smem = static_cast<size_t>(R_WARPS + 1) * E * 4;   // at most 36 KB
        with_row_shape(E, whole_vectors(E, logits, nullptr), [&](auto v, auto l, auto n) {
            balance_partial_kernel<v.value, l.value, n.value><<<ch.count, R_THREADS, smem, s>>>(
                logits, topk_idx, token_mask, seq_offsets, S, T, E, k, ch.per, psum, pcnt, pn,
                dev_status);
        });
        if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    }
    balance_combine_kernel<<<C_CTAS, R_THREADS, 0, s>>>(psum, pcnt, pn, seq_offsets, S, T, E, k,
                                                        ch.per, coef, loss, counts, prob_mean,
                                                        n_tokens, dev_status);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status_t moe_gate_topk_backward(
    const float *logits, const int32_t *topk_idx, const float *d_topk_w, const uint8_t *token_mask,
    const int32_t *seq_offsets, int32_t S, const int32_t *counts, const int32_t *n_tokens,
    const float *d_loss, float coef, int32_t T, int32_t E, int32_t k, uint32_t flags,
    float *d_logits, int32_t *dev_status, moe_stream_t stream) {
    if (T < 0 || E <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (E > 1024 || k > 32 || k > E) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(T) * k >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!counts != !n_tokens) return MOE_ERR_INVALID_ARG;
    if (counts && (S <= 0 || (!seq_offsets && S != 1))) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!logits || !d_logits || (d_topk_w && !topk_idx)) return MOE_ERR_INVALID_ARG;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Chunks ch = chunks_of(T);
    with_row_shape(E, whole_vectors(E, logits, d_logits), [&](auto v, auto l, auto n) {
        topk_backward_kernel<v.value, l.value, n.value><<<ch.count, R_THREADS, 0, s>>>(
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
    const int grid = static_cast<int>(std::min<int64_t>(units, static_cast<int64_t>(num_sms()) * 16));
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
