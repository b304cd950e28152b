// norm.cu -- what stands between two blocks of a residual stream: the norm
// after a block with its gate and residual scale, the addition, and the norm
// before the next block, in one pass each way.
//
//   N(v; gamma) = gamma k v,  k = 1 / sqrt(mean(v^2) + eps)
//   r  = x + scale gate[s] N(y; gamma_post),   xn = N(r; gamma_next)
// for the tokens of sequence s.  Backward, with r^ = k_r r, y^ = k_y y, t = d_xn
// gamma_next and means over a row:
//   d   = d_r + k_r (t - r^ mean(t r^))                    (the gradient of x)
//   q   = scale d gate[s] gamma_post
//   d_y = k_y (q - y^ mean(q y^))
//   c[s] = sum over s of scale d y^:  d_gate[s] = gamma_post c[s],
//   d_gamma_post = sum_s gate[s] c[s],   d_gamma_next = sum d_xn r^
//
// What bounds it is memory: every row is read and written once.  A team of 1 to 8
// warps takes a row (8 columns a lane and step); rows come through a ring of
// shared-memory slots filled by bulk copies some rows ahead, so that the copies
// run on through the two sums a row waits for (one barrier each).  A team takes
// consecutive rows and keeps the column sums in registers; it writes them out
// when a sequence ends, team i's sums of sequence s to slot i + s (both only
// grow along the rows, so no two meet), and a second kernel adds the slots in a
// fixed order.
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CTAS = 304;             // two on each of 152 multiprocessors
constexpr int MAX_SLOTS = 4;
constexpr int MAX_H = 8192;

// Layout of rows of H columns: warps per team, teams per CTA, vectors per lane.
struct Shape {
    int W, teams, vpt;
};
__host__ __device__ inline Shape shape_of(int H) {
    const int need = (H / 8 + 31) / 32;
    Shape s;
    s.W = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : 8;
    s.teams = WARPS / s.W;
    const int v = (need + s.W - 1) / s.W;
    s.vpt = v <= 1 ? 1 : v <= 2 ? 2 : 4;
    return s;
}
inline int teams_of(int T, int H) {
    return static_cast<int>(std::min<int64_t>(T, static_cast<int64_t>(MAX_CTAS) * shape_of(H).teams));
}

struct Params {
    // ring arrays: forward y, x; backward d_xn, r, d_r, y (NULL: absent)
    const void *src[4];
    const uint16_t *gamma_post, *gate, *gamma_next;
    const int32_t *seq;
    int32_t S;                 // sequences (1 without a gate)
    int32_t T, H;
    float scale, eps;
    int32_t post;              // the norm after the block
    int32_t next;              // the norm before the next one
    int32_t nteams, slots;
    int32_t slot_bytes;        // of one row's arrays
    int32_t off[4];            // of each array in a slot
    int32_t bytes[4];
    void *out0, *out1;         // forward r, xn; backward d_x, d_y
    float *rstd_post, *rstd_next;
    const float *k_post, *k_next;
    float *part_c, *part_n;    // column sums: [nteams + S][H], [nteams][H] (NULL: not wanted)
    int32_t *dev_status;
};

template <bool F32>
__device__ __forceinline__ void load8(const void *base, int v, float (&o)[8]) {
    if (F32) {
        const float4 a = reinterpret_cast<const float4 *>(base)[2 * v];
        const float4 b = reinterpret_cast<const float4 *>(base)[2 * v + 1];
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
        o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    } else {
        const uint4 q = reinterpret_cast<const uint4 *>(base)[v];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(w[i] << 16);
            o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ void unpack8(const uint4 &q, float (&o)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&o)[8]) {
    return make_uint4(bf16x2(o[0], o[1]), bf16x2(o[2], o[3]), bf16x2(o[4], o[5]), bf16x2(o[6], o[7]));
}
template <bool F32>
__device__ __forceinline__ void store8(void *row, int v, const float (&o)[8]) {
    if (F32) {
        __stcs(reinterpret_cast<float4 *>(row) + 2 * v, make_float4(o[0], o[1], o[2], o[3]));
        __stcs(reinterpret_cast<float4 *>(row) + 2 * v + 1, make_float4(o[4], o[5], o[6], o[7]));
    } else {
        __stcs(reinterpret_cast<uint4 *>(row) + v, pack8(o));
    }
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// A team: its threads' sum of a value (each call another of two buffers, so
// one barrier a call is enough).
struct Team {
    int W, id, lane, warp;      // warps, number in the CTA, lane and warp in the team
    float *red;                 // [2][WARPS]
    int parity;
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (W == 1) return v;
        float *b = red + parity * WARPS;
        parity ^= 1;
        if (lane == 0) b[warp] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(32 * W) : "memory");
        float s = 0.0f;
        for (int i = 0; i < W; ++i) s += b[i];
        return s;
    }
};

// Sequence of row t; -1 in front of the first one.
__device__ __forceinline__ int find_sequence(const int32_t *seq, int S, int t) {
    int lo = -1, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(seq + mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// False where the bounds do not ascend inside [0, T].  All threads of the CTA.
__device__ bool bounds_ok(const Params &p) {
    int bad = 0;
    if (p.seq)
        for (int s = threadIdx.x; s <= p.S; s += THREADS) {
            const int a = __ldg(p.seq + s);
            bad |= a < 0 || a > p.T || (s < p.S && __ldg(p.seq + s + 1) < a);
        }
    return !__syncthreads_or(bad);
}

// The rows of a team, one after the other: body(row, sequence, slot's address).
// `body` calls the team's barrier at least once after its last read of the slot
// and then release().
template <bool BWD, bool XF, bool YF, int VPT>
__global__ void __launch_bounds__(THREADS, VPT <= 2 ? 2 : 1) norm_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_bar[WARPS][MAX_SLOTS];
    __shared__ float s_red[WARPS][2][WARPS];
    __shared__ int s_abort;
    const Shape sh = shape_of(p.H);
    const int warp = threadIdx.x >> 5;
    Team team;
    team.W = sh.W;
    team.id = warp / sh.W;
    team.warp = warp % sh.W;
    team.lane = threadIdx.x & 31;
    team.red = &s_red[team.id][0][0];
    team.parity = 0;
    const int me = team.warp * 32 + team.lane, size = 32 * sh.W;
    const bool first = me == 0;
    uint8_t *ring = smem + team.id * p.slots * p.slot_bytes;
    uint64_t *bar = s_bar[team.id];
    if (first) {
        for (int i = 0; i < p.slots; ++i) mbar_init(&bar[i], 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) s_abort = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool good = bounds_ok(p);                  // (its barrier publishes the mbarriers)
    if (!good) {
        if (threadIdx.x == 0 && blockIdx.x == 0) report(p.dev_status, MOE_DEV_BAD_OFFSETS);
        return;
    }
    const int t_id = blockIdx.x * sh.teams + team.id;
    if (t_id >= p.nteams) return;
    int a = static_cast<int>(static_cast<int64_t>(t_id) * p.T / p.nteams);
    int b = static_cast<int>(static_cast<int64_t>(t_id + 1) * p.T / p.nteams);
    if (p.seq) {                                     // rows outside every sequence are left alone
        a = max(a, __ldg(p.seq));
        b = min(b, __ldg(p.seq + p.S));
    }
    volatile int *abort = &s_abort;

    int fetched = 0;                                 // rows asked for (the first thread's count)
    auto fetch = [&](int row, int slot) {
        ++fetched;
        mbar_arrive_expect_tx(&bar[slot], static_cast<uint32_t>(p.slot_bytes));
#pragma unroll
        for (int i = 0; i < (BWD ? 4 : 2); ++i)
            if (p.src[i])
                bulk_load(ring + slot * p.slot_bytes + p.off[i],
                          static_cast<const uint8_t *>(p.src[i]) + static_cast<int64_t>(row) * p.bytes[i],
                          static_cast<uint32_t>(p.bytes[i]), &bar[slot]);
    };
    if (first)
        for (int i = 0; i < p.slots && a + i < b; ++i) fetch(a + i, i);

    const int nvec = p.H / 8;
    const float inv_h = 1.0f / static_cast<float>(p.H);
    int seq = p.seq && a < b ? find_sequence(p.seq, p.S, a) : 0;
    int seq_end = p.seq && a < b ? __ldg(p.seq + seq + 1) : p.T;
    // the gammas and the gate of this lane's columns
    uint4 gp[VPT], gn[VPT], gt[VPT];
    const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    auto gate_row = [&]() {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = me + j * size;
            gt[j] = p.gate && v < nvec
                        ? __ldg(reinterpret_cast<const uint4 *>(p.gate) + static_cast<int64_t>(seq) * nvec + v)
                        : ones;
        }
    };
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = me + j * size;
        gp[j] = p.gamma_post && v < nvec ? __ldg(reinterpret_cast<const uint4 *>(p.gamma_post) + v) : ones;
        gn[j] = p.gamma_next && v < nvec ? __ldg(reinterpret_cast<const uint4 *>(p.gamma_next) + v) : ones;
    }
    if (a < b) gate_row();
    float cs[BWD ? VPT : 1][8], ns[BWD ? VPT : 1][8];
    auto clear = [&](float (&s)[BWD ? VPT : 1][8]) {
#pragma unroll
        for (int j = 0; j < (BWD ? VPT : 1); ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j][i] = 0.0f;
    };
    auto flush = [&](float *part, int64_t slot, const float (&s)[BWD ? VPT : 1][8]) {
        if (!part) return;
#pragma unroll
        for (int j = 0; j < (BWD ? VPT : 1); ++j) {
            const int v = me + j * size;
            if (v >= nvec) continue;
            float4 *d = reinterpret_cast<float4 *>(part + slot * p.H) + 2 * v;
            d[0] = make_float4(s[j][0], s[j][1], s[j][2], s[j][3]);
            d[1] = make_float4(s[j][4], s[j][5], s[j][6], s[j][7]);
        }
    };
    clear(cs);
    clear(ns);

    int slot = 0;
    uint32_t phase = 0;
    for (int row = a; row < b; ++row) {
        if (row == seq_end) {                        // the next sequence that has rows
            if (BWD) {
                flush(p.part_c, t_id + seq, cs);
                clear(cs);
            }
            do
                seq_end = __ldg(p.seq + ++seq + 1);
            while (seq_end == row);
            gate_row();
        }
        const uint8_t *in = ring + slot * p.slot_bytes;
        mbar_wait_bounded(&bar[slot], phase, abort, p.dev_status);
        const bool keep = *abort == 0;
        auto release = [&]() {
            if (first && row + p.slots < b && *abort == 0) fetch(row + p.slots, slot);
        };
        if (!BWD) {
            const void *ys = in + p.off[0], *xs = in + p.off[1];
            float ky = 1.0f;
            if (p.post) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = me + j * size;
                    if (v >= nvec) continue;
                    float y[8];
                    load8<YF>(ys, v, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
                }
                ky = 1.0f / sqrtf(team.sum(ss) * inv_h + p.eps);
                if (first && keep && p.rstd_post) p.rstd_post[row] = ky;
            }
            float r[VPT][8], ss = 0.0f;
            uint8_t *ro = static_cast<uint8_t *>(p.out0) + static_cast<int64_t>(row) * p.H * (XF ? 4 : 2);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = me + j * size;
                if (v >= nvec) continue;
                float y[8], x[8], g[8], f[8];
                load8<YF>(ys, v, y);
                load8<XF>(xs, v, x);
                unpack8(gt[j], g);
                unpack8(gp[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[j][i] = fmaf(p.scale * g[i], y[i] * ky * f[i], x[i]);
                if (!XF) unpack8(pack8(r[j]), r[j]);     // the norm of what is stored
                if (keep) store8<XF>(ro, v, r[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(r[j][i], r[j][i], ss);
            }
            const float tot = team.sum(ss);
            if (team.W == 1) __syncwarp();
            release();
            if (p.next) {
                const float kr = 1.0f / sqrtf(tot * inv_h + p.eps);
                if (first && keep && p.rstd_next) p.rstd_next[row] = kr;
                uint8_t *xo = static_cast<uint8_t *>(p.out1) + static_cast<int64_t>(row) * p.H * 2;
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = me + j * size;
                    if (v >= nvec) continue;
                    float f[8], o[8];
                    unpack8(gn[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = r[j][i] * kr * f[i];
                    if (keep) store8<false>(xo, v, o);
                }
            }
        } else {
            const void *nx = in + p.off[0], *rs = in + p.off[1], *dr = in + p.off[2], *ys = in + p.off[3];
            float m1 = 0.0f, kr = 0.0f;
            if (p.next) {
                kr = __ldg(p.k_next + row);
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = me + j * size;
                    if (v >= nvec) continue;
                    float d[8], r[8], f[8];
                    load8<false>(nx, v, d);
                    load8<XF>(rs, v, r);
                    unpack8(gn[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float dr_hat = d[i] * (r[i] * kr);
                        ns[j][i] += dr_hat;
                        m1 = fmaf(dr_hat, f[i], m1);
                    }
                }
                m1 = team.sum(m1) * inv_h;
            }
            const float ky = p.post ? __ldg(p.k_post + row) : 1.0f;
            float q[VPT][8], yh[VPT][8], m2 = 0.0f;
            uint8_t *xo = static_cast<uint8_t *>(p.out0) + static_cast<int64_t>(row) * p.H * (XF ? 4 : 2);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = me + j * size;
                if (v >= nvec) continue;
                float d[8], f[8], g[8];
                if (p.src[2])
                    load8<XF>(dr, v, d);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] = 0.0f;
                if (p.next) {
                    float t[8], r[8];
                    load8<false>(nx, v, t);
                    load8<XF>(rs, v, r);
                    unpack8(gn[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[i] = fmaf(kr, fmaf(-(r[i] * kr), m1, t[i] * f[i]), d[i]);
                }
                if (keep && p.out0) store8<XF>(xo, v, d);
                load8<YF>(ys, v, yh[j]);
                unpack8(gt[j], g);
                unpack8(gp[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    yh[j][i] *= ky;
                    const float sd = p.scale * d[i];
                    cs[j][i] = fmaf(sd, yh[j][i], cs[j][i]);
                    q[j][i] = sd * g[i] * f[i];
                    m2 = fmaf(q[j][i], yh[j][i], m2);
                }
            }
            m2 = team.sum(m2) * inv_h;
            if (team.W == 1) __syncwarp();
            release();
            if (!p.post) m2 = 0.0f;
            uint8_t *yo = static_cast<uint8_t *>(p.out1) + static_cast<int64_t>(row) * p.H * (YF ? 4 : 2);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = me + j * size;
                if (v >= nvec) continue;
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = ky * fmaf(-yh[j][i], m2, q[j][i]);
                if (keep && p.out1) store8<YF>(yo, v, o);
            }
        }
        if (++slot == p.slots) {
            slot = 0;
            phase ^= 1;
        }
    }
    if (BWD) {
        if (a < b) flush(p.part_c, t_id + seq, cs);
        flush(p.part_n, t_id, ns);
    }
    if (first && *abort)                             // copies still on their way land first
        for (int i = max(0, fetched - p.slots); i < fetched; ++i)
            mbar_wait_drain(&bar[i % p.slots], static_cast<uint32_t>(i / p.slots) & 1u);
}

// Adds up the teams' column sums: 32 columns per CTA.  With few sequences all
// warps share the teams of one, with many (16 or more) each takes sequences of
// its own.
constexpr int RED_WARPS = 16;
struct SumParams {
    const float *part_c, *part_n;
    const uint16_t *gamma_post, *gate;
    const int32_t *seq;
    int32_t S, T, H, nteams;
    float *d_gamma_post, *d_gate, *d_gamma_next;
};
__device__ __forceinline__ float add_slots(const float *part, int64_t slot0, int n, int first, int step,
                                           int H, int col) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int i = first;
    for (; i + 3 * step < n; i += 4 * step)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] += __ldg(part + (slot0 + i + k * step) * H + col);
    for (; i < n; i += step) s[0] += __ldg(part + (slot0 + i) * H + col);
    return (s[0] + s[1]) + (s[2] + s[3]);
}
__global__ void __launch_bounds__(32 * RED_WARPS) norm_sums_kernel(const SumParams p) {
    __shared__ float s_red[RED_WARPS][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int bad = 0;                                     // bounds as the first kernel judged them
    if (p.seq)
        for (int s = threadIdx.x; s <= p.S; s += 32 * RED_WARPS) {
            const int a = __ldg(p.seq + s);
            bad |= a < 0 || a > p.T || (s < p.S && __ldg(p.seq + s + 1) < a);
        }
    if (__syncthreads_or(bad)) return;
    const int h = blockIdx.x * 32 + lane;
    const int col = min(h, p.H - 1);
    const bool in = h < p.H;
    auto bf = [&](const uint16_t *v, int64_t i) { return v ? bf16_bits_to_float(__ldg(v + i)) : 1.0f; };
    auto block_sum = [&](float v) {
        s_red[warp][lane] = v;
        __syncthreads();
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < RED_WARPS; ++w) s += s_red[w][lane];
        __syncthreads();
        return s;
    };
    // the teams that have rows of [a, b): team i owns rows [i T / n, (i + 1) T / n)
    auto team_of = [&](int row) {
        int i = static_cast<int>((static_cast<int64_t>(row) * p.nteams) / p.T);
        while (static_cast<int64_t>(i + 1) * p.T / p.nteams <= row) ++i;
        while (static_cast<int64_t>(i) * p.T / p.nteams > row) --i;
        return i;
    };
    if (p.d_gamma_next) {
        const float v = block_sum(add_slots(p.part_n, 0, p.nteams, warp, RED_WARPS, p.H, col));
        if (warp == 0 && in) p.d_gamma_next[h] = v;
    }
    if (!p.d_gamma_post && !p.d_gate) return;
    const float gp = bf(p.gamma_post, col);
    float gamma = 0.0f;
    const bool shared = p.S < RED_WARPS;
    for (int s = shared ? 0 : warp; s < p.S; s += shared ? 1 : RED_WARPS) {
        const int a = p.seq ? __ldg(p.seq + s) : 0, b = p.seq ? __ldg(p.seq + s + 1) : p.T;
        float c = 0.0f;
        if (a < b) {
            const int t0 = team_of(a), t1 = team_of(b - 1);
            c = add_slots(p.part_c, static_cast<int64_t>(t0) + s, t1 - t0 + 1, shared ? warp : 0,
                          shared ? RED_WARPS : 1, p.H, col);
        }
        if (shared) c = block_sum(c);
        if (p.d_gate && in && (!shared || warp == 0)) p.d_gate[static_cast<int64_t>(s) * p.H + h] = gp * c;
        gamma = fmaf(bf(p.gate, static_cast<int64_t>(s) * p.H + col), c, gamma);
    }
    if (p.d_gamma_post) {
        if (!shared) gamma = block_sum(gamma);
        if (warp == 0 && in) p.d_gamma_post[h] = gamma;
    }
}

// ------------------------------------------------------------------ host side
inline bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename K, typename P>
cudaError_t start(K kernel, int grid, int block, int smem, const P &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(block), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool BWD, bool XF, bool YF, int VPT>
cudaError_t launch_shape(const Params &p, const Shape &sh, cudaStream_t stream) {
    auto kernel = norm_kernel<BWD, XF, YF, VPT>;
    constexpr int MAX_SMEM = 224 * 1024;
    static std::mutex mu;
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !attr_done[dev]) {
            const cudaError_t e =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
            if (e != cudaSuccess) return e;
            if (dev < 64) attr_done[dev] = true;
        }
    }
    const int grid = static_cast<int>(ceil_div(p.nteams, sh.teams));
    return start(kernel, grid, THREADS, sh.teams * p.slots * p.slot_bytes, p, stream);
}

template <bool BWD>
cudaError_t launch(Params &p, bool xf, bool yf, cudaStream_t stream) {
    const Shape sh = shape_of(p.H);
    p.nteams = teams_of(p.T, p.H);
    int at = 0;
    for (int i = 0; i < 4; ++i) {
        p.off[i] = at;
        if (p.src[i]) at += p.bytes[i];
    }
    p.slot_bytes = at;
    // rows ahead: as many as two CTAs a multiprocessor have room for, or one where
    // that is less than two
    const int row = sh.teams * at;
    p.slots = std::min(MAX_SLOTS, 104 * 1024 / row);
    if (p.slots < 2) p.slots = std::max(1, std::min(MAX_SLOTS, 208 * 1024 / row));
#define MOE_NORM(X, Y)                                                                        \
    (sh.vpt == 1   ? launch_shape<BWD, X, Y, 1>(p, sh, stream)                               \
     : sh.vpt == 2 ? launch_shape<BWD, X, Y, 2>(p, sh, stream)                               \
                   : launch_shape<BWD, X, Y, 4>(p, sh, stream))
    if (xf) return yf ? MOE_NORM(true, true) : MOE_NORM(true, false);
    return yf ? MOE_NORM(false, true) : MOE_NORM(false, false);
#undef MOE_NORM
}

moe_status_t check_sizes(int32_t T, int32_t H, int32_t S) {
    if (T < 0 || H <= 0 || S <= 0) return MOE_ERR_INVALID_ARG;
    if (H % 8 != 0 || H > MAX_H || T > (1 << 30) || S > 65536) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

size_t part_bytes(int64_t slots, int H) {
    return (static_cast<size_t>(slots) * H * 4 + 255) & ~static_cast<size_t>(255);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_norm_residual(const void *x, const void *y, const moe_bf16_t *gamma_post,
                                          const moe_bf16_t *gate, const int32_t *seq_offsets, int32_t S,
                                          const moe_bf16_t *gamma_next, int32_t T, int32_t H, float scale,
                                          float eps, uint32_t flags, void *r, moe_bf16_t *xn,
                                          float *rstd_post, float *rstd_next, int32_t *dev_status,
                                          moe_stream_t stream) {
    if (!gate) {
        seq_offsets = nullptr;
        S = 1;
    }
    const moe_status_t st = check_sizes(T, H, S);
    if (st != MOE_OK) return st;
    const bool xf = (flags & MOE_RES_F32) != 0, yf = (flags & MOE_Y_F32) != 0;
    const bool post = (flags & MOE_POST_NORM) != 0;
    if ((!seq_offsets && S != 1) || (!post && gamma_post) || (!xn && (gamma_next || rstd_next)))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !y || !r || !a16(x) || !a16(y) || !a16(r) || !a16(xn) || !a16(gamma_post) || !a16(gate) ||
        !a16(gamma_next))
        return MOE_ERR_INVALID_ARG;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    Params p{};
    p.src[0] = y;
    p.bytes[0] = H * (yf ? 4 : 2);
    p.src[1] = x;
    p.bytes[1] = H * (xf ? 4 : 2);
    p.gamma_post = gamma_post;
    p.gate = gate;
    p.gamma_next = gamma_next;
    p.seq = seq_offsets;
    p.S = S;
    p.T = T;
    p.H = H;
    p.scale = scale;
    p.eps = eps;
    p.post = post;
    p.next = xn != nullptr;
    p.out0 = r;
    p.out1 = xn;
    p.rstd_post = post ? rstd_post : nullptr;
    p.rstd_next = rstd_next;
    p.dev_status = dev_status;
    return launch<false>(p, xf, yf, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                           : MOE_ERR_CUDA;
}

extern "C" moe_status_t moe_norm_residual_backward_workspace_size(int32_t T, int32_t H, int32_t S,
                                                                  size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_sizes(T, H, S);
    if (st != MOE_OK) return st;
    const int64_t n = teams_of(T, H);
    *bytes = part_bytes(n + S, H) + part_bytes(n, H);
    return MOE_OK;
}

extern "C" moe_status_t moe_norm_residual_backward(
    const void *d_r, const moe_bf16_t *d_xn, const void *y, const void *r, const float *rstd_post,
    const float *rstd_next, const moe_bf16_t *gamma_post, const moe_bf16_t *gate,
    const int32_t *seq_offsets, int32_t S, const moe_bf16_t *gamma_next, int32_t T, int32_t H, float scale,
    uint32_t flags, void *d_x, void *d_y, float *d_gamma_post, float *d_gate, float *d_gamma_next,
    void *workspace, size_t workspace_bytes, int32_t *dev_status, moe_stream_t stream) {
    if (!gate) {
        seq_offsets = nullptr;
        S = 1;
    }
    const moe_status_t st = check_sizes(T, H, S);
    if (st != MOE_OK) return st;
    const bool xf = (flags & MOE_RES_F32) != 0, yf = (flags & MOE_Y_F32) != 0;
    const bool post = (flags & MOE_POST_NORM) != 0;
    if ((!seq_offsets && S != 1) || (!post && (gamma_post || d_gamma_post)) || (!gate && d_gate))
        return MOE_ERR_INVALID_ARG;
    const bool sums = d_gamma_post || d_gate, any = sums || d_gamma_next;
    if (T > 0) {                                     // (no rows may come as no pointers)
        if ((!d_xn && (gamma_next || d_gamma_next)) || (!d_r && !d_xn)) return MOE_ERR_INVALID_ARG;
        if (!y || (post && !rstd_post) || (d_xn && (!r || !rstd_next))) return MOE_ERR_INVALID_ARG;
        if (!a16(d_r) || !a16(d_xn) || !a16(y) || !a16(r) || !a16(gamma_post) || !a16(gate) ||
            !a16(gamma_next) || !a16(d_x) || !a16(d_y))
            return MOE_ERR_INVALID_ARG;
        size_t need = 0;
        moe_norm_residual_backward_workspace_size(T, H, S, &need);
        if (any && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)))
            return MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        const size_t row = static_cast<size_t>(H) * 4;
        if ((d_gamma_post && cudaMemsetAsync(d_gamma_post, 0, row, s) != cudaSuccess) ||
            (d_gate && cudaMemsetAsync(d_gate, 0, row * S, s) != cudaSuccess) ||
            (d_gamma_next && cudaMemsetAsync(d_gamma_next, 0, row, s) != cudaSuccess))
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    Params p{};
    p.src[0] = d_xn;
    p.bytes[0] = H * 2;
    p.src[1] = d_xn ? r : nullptr;
    p.bytes[1] = H * (xf ? 4 : 2);
    p.src[2] = d_r;
    p.bytes[2] = H * (xf ? 4 : 2);
    p.src[3] = y;
    p.bytes[3] = H * (yf ? 4 : 2);
    p.gamma_post = gamma_post;
    p.gate = gate;
    p.gamma_next = gamma_next;
    p.seq = seq_offsets;
    p.S = S;
    p.T = T;
    p.H = H;
    p.scale = scale;
    p.post = post;
    p.next = d_xn != nullptr;
    p.out0 = d_x;
    p.out1 = d_y;
    p.k_post = rstd_post;
    p.k_next = rstd_next;
    p.dev_status = dev_status;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const int n = teams_of(T, H);
    if (sums) p.part_c = reinterpret_cast<float *>(ws);
    if (d_gamma_next)
        p.part_n = reinterpret_cast<float *>(ws + part_bytes(static_cast<int64_t>(n) + S, H));
    if (launch<true>(p, xf, yf, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (!any) return MOE_OK;
    SumParams q{};
    q.part_c = p.part_c;
    q.part_n = p.part_n;
    q.gamma_post = gamma_post;
    q.gate = gate;
    q.seq = seq_offsets;
    q.S = S;
    q.T = T;
    q.H = H;
    q.nteams = p.nteams;
    q.d_gamma_post = d_gamma_post;
    q.d_gate = d_gate;
    q.d_gamma_next = d_gamma_next;
    if (start(norm_sums_kernel, static_cast<int>(ceil_div(H, 32)), 32 * RED_WARPS, 0, q, s) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}
