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
// run on through the sums a row waits for (its second one and the next row's first
// share a barrier: 144 us backward where two took 211).  A team takes
// consecutive rows and keeps the column sums in registers; it writes them out
// when a sequence ends, team i's sums of sequence s to slot i + s (both only
// grow along the rows, so no two meet), and a second kernel adds the slots in a
// fixed order.  16384 rows of 4096, bf16: 89 us forward (6.0 TB/s), 143 backward (5.6);
// 50021 of 2048 with an fp32 stream: 308 backward (6.0); 16384 of 8192, bf16: 183 and 260
// (5.9 and 6.2).  One row: 3.7.
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
// two on each of 152 multiprocessors; rows of more than 4096 columns leave room for one
// (their registers), and those CTAs run in two rounds
constexpr int MAX_CTAS = 304;
constexpr int MAX_SLOTS = 4;
constexpr int MAX_H = 8192;
constexpr int MAX_SMEM = 224 * 1024;      // two rows of 8192 columns, all arrays fp32 that can be

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

// Eight values as four pairs: of a bf16 vector, or the v-th eight of a row.
__device__ __forceinline__ void widen(const uint4 &q, f2 (&o)[4]) {
    o[0] = from_bf16x2(q.x), o[1] = from_bf16x2(q.y);
    o[2] = from_bf16x2(q.z), o[3] = from_bf16x2(q.w);
}
template <bool F32>
__device__ __forceinline__ void load8(const void *base, int v, f2 (&o)[4]) {
    if (F32) {
        const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(base)[2 * v];
        const ulonglong2 b = reinterpret_cast<const ulonglong2 *>(base)[2 * v + 1];
        o[0] = a.x, o[1] = a.y, o[2] = b.x, o[3] = b.y;
    } else {
        widen(reinterpret_cast<const uint4 *>(base)[v], o);
    }
}
__device__ __forceinline__ uint4 narrow(const f2 (&o)[4]) {
    return make_uint4(to_bf16x2(o[0]), to_bf16x2(o[1]), to_bf16x2(o[2]), to_bf16x2(o[3]));
}
template <bool F32>
__device__ __forceinline__ void store8(void *row, int v, const f2 (&o)[4]) {
    if (F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 a = unpack2(o[2 * i]), b = unpack2(o[2 * i + 1]);
            __stcs(reinterpret_cast<float4 *>(row) + 2 * v + i, make_float4(a.x, a.y, b.x, b.y));
        }
    } else {
        __stcs(reinterpret_cast<uint4 *>(row) + v, narrow(o));
    }
}
__device__ __forceinline__ float total2(f2 v) {
    const float2 f = unpack2(v);
    return f.x + f.y;
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// A team: its threads' sums of two values (each call another of two buffers, so
// one barrier a call is enough).
struct Team {
    int W, id, lane, warp;      // warps, number in the CTA, lane and warp in the team
    float2 *red;                // [2][WARPS]
    int parity;
    __device__ __forceinline__ float2 sum(float x, float y) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, off);
            y += __shfl_xor_sync(0xffffffffu, y, off);
        }
        if (W == 1) {
            __syncwarp();
            return make_float2(x, y);
        }
        float2 *b = red + parity * WARPS;
        parity ^= 1;
        if (lane == 0) b[warp] = make_float2(x, y);
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(32 * W) : "memory");
        float2 s = make_float2(0.0f, 0.0f);
        for (int i = 0; i < W; ++i) {
            s.x += b[i].x;
            s.y += b[i].y;
        }
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

template <bool BWD, bool XF, bool YF, int VPT>
__global__ void __launch_bounds__(THREADS, VPT <= 2 ? 2 : 1) norm_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_bar[WARPS][MAX_SLOTS];
    __shared__ float2 s_red[WARPS][2][WARPS];
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
    // What a lane keeps of its columns: gamma_next, and scale * gate * gamma_post
    // (without the scale in the backward pass, where it joins a row's factor)
    uint4 gn[VPT];
    f2 gf[VPT][4];
    const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    auto column = [&](const uint16_t *base, int64_t row, int v) {
        return base && v < nvec ? __ldg(reinterpret_cast<const uint4 *>(base) + row * nvec + v) : ones;
    };
    auto gate_row = [&]() {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = me + j * size;
            f2 g[4], f[4];
            widen(column(p.gate, seq, v), g);
            widen(column(p.gamma_post, 0, v), f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                gf[j][i] = mul2(g[i], f[i]);
                if (!BWD) gf[j][i] = mul2(gf[j][i], splat(p.scale));
            }
        }
    };
#pragma unroll
    for (int j = 0; j < VPT; ++j) gn[j] = column(p.gamma_next, 0, me + j * size);
    if (a < b) gate_row();
    constexpr int AV = BWD ? VPT : 1;
    f2 cs[AV][4], ns[AV][4];
    auto clear = [&](f2 (&s)[AV][4]) {
#pragma unroll
        for (int j = 0; j < AV; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] = 0;
    };
    auto flush = [&](float *part, int64_t slot, const f2 (&s)[AV][4]) {
        if (!part) return;
#pragma unroll
        for (int j = 0; j < AV; ++j) {
            const int v = me + j * size;
            if (v >= nvec) continue;
            ulonglong2 *d = reinterpret_cast<ulonglong2 *>(part + slot * p.H) + 2 * v;
            d[0] = make_ulonglong2(s[j][0], s[j][1]);
            d[1] = make_ulonglong2(s[j][2], s[j][3]);
        }
    };
    clear(cs);
    clear(ns);

    // A row's two sums depend on one another, but the second one of a row and the
    // first one of the next do not: they are taken together, one barrier a row.
    int slot = 0;
    uint32_t phase = 0;
    const uint8_t *in = ring;
    bool keep = true;                                // no wait has given up
    auto arrive = [&]() {                            // the row in `slot` has landed
        in = ring + slot * p.slot_bytes;
        mbar_wait_bounded(&bar[slot], phase, abort, p.dev_status);
        keep = *abort == 0;
    };
    const f2 ks2 = splat(p.scale);
    // first sum of a row: forward of y^2; backward of w r with w = k_r d_xn gamma_next
    // (and the column sums of d_xn r^)
    auto first_sum = [&](float k_next) {
        f2 m = 0;
        if (BWD ? p.next : p.post) {
            const f2 kr2 = splat(k_next);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = me + j * size;
                if (v >= nvec) continue;
                if (!BWD) {
                    f2 y[4];
                    load8<YF>(in + p.off[0], v, y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) m = fma2(y[i], y[i], m);
                } else {
                    f2 d[4], r[4], f[4];
                    load8<false>(in + p.off[0], v, d);
                    load8<XF>(in + p.off[1], v, r);
                    widen(gn[j], f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f2 u = mul2(d[i], kr2);
                        ns[j % AV][i] = fma2(u, r[i], ns[j % AV][i]);
                        m = fma2(mul2(u, f[i]), r[i], m);
                    }
                }
            }
        }
        return total2(m);
    };
    float k_next = 0.0f, s1 = 0.0f;
    if (a < b) {
        if (BWD && p.next) k_next = __ldg(p.k_next + a);
        arrive();
        s1 = team.sum(first_sum(k_next), 0.0f).x;
    }
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
        const bool more = row + 1 < b;
        const int this_slot = slot;
        const float k_post = BWD && p.post ? __ldg(p.k_post + row) : 1.0f;
        const float k_after = BWD && p.next && more ? __ldg(p.k_next + row + 1) : 0.0f;
        f2 keep_q[VPT][4], m = 0;                    // forward r, backward q
        uint4 yq[BWD && !YF ? VPT : 1];
        f2 yf[BWD && YF ? VPT : 1][4];
        if (!BWD) {
            float ky = 1.0f;
            if (p.post) {
                ky = 1.0f / sqrtf(s1 * inv_h + p.eps);
                if (first && keep && p.rstd_post) p.rstd_post[row] = ky;
            }
            const f2 ky2 = splat(ky);
            uint8_t *ro = static_cast<uint8_t *>(p.out0) + static_cast<int64_t>(row) * p.H * (XF ? 4 : 2);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = me + j * size;
                if (v >= nvec) continue;
                f2 y[4], x[4];
                load8<YF>(in + p.off[0], v, y);
                load8<XF>(in + p.off[1], v, x);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = fma2(mul2(y[i], ky2), gf[j][i], x[i]);
                if (XF) {
                    if (keep) store8<true>(ro, v, x);
                } else {                             // the norm is that of what is stored
                    const uint4 q = narrow(x);
                    if (keep) __stcs(reinterpret_cast<uint4 *>(ro) + v, q);
                    widen(q, x);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    m = fma2(x[i], x[i], m);
                    keep_q[j][i] = x[i];
                }
            }
        } else {
            // With the row factors taken out of the sums,
            //   d = d_r + w - r (k_r^2 mean(w r)),
            // and, with q = scale k_y d gate gamma_post, d_y = q - y (k_y^2 mean(q y)).
            const f2 kr2 = splat(k_next), ky2 = mul2(ks2, splat(k_post));
            const f2 c1 = splat(-k_next * k_next * (s1 * inv_h));
            uint8_t *xo = static_cast<uint8_t *>(p.out0) + static_cast<int64_t>(row) * p.H * (XF ? 4 : 2);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = me + j * size;
                if (v >= nvec) continue;
                f2 d[4];
                if (p.src[2])
                    load8<XF>(in + p.off[2], v, d);
                else
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = 0;
                if (p.next) {
                    f2 t[4], r[4], f[4];
                    load8<false>(in + p.off[0], v, t);
                    load8<XF>(in + p.off[1], v, r);
                    widen(gn[j], f);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        d[i] = fma2(r[i], c1, fma2(mul2(t[i], kr2), f[i], d[i]));
                }
                if (keep && p.out0) store8<XF>(xo, v, d);
                f2 y[4];
                if (YF) {
                    load8<true>(in + p.off[3], v, yf[YF ? j : 0]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = yf[YF ? j : 0][i];
                } else {
                    yq[YF ? 0 : j] = reinterpret_cast<const uint4 *>(in + p.off[3])[v];
                    widen(yq[YF ? 0 : j], y);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f2 e = mul2(d[i], ky2);
                    cs[j % AV][i] = fma2(e, y[i], cs[j % AV][i]);
                    keep_q[j][i] = mul2(e, gf[j][i]);
                    m = fma2(keep_q[j][i], y[i], m);
                }
            }
        }
        float ahead = 0.0f;
        if (more) {
            if (++slot == p.slots) {
                slot = 0;
                phase ^= 1;
            }
            arrive();
            ahead = first_sum(k_after);
        }
        fence_proxy_async();                         // (reads, before the slot is filled again)
        const float2 sums = team.sum(total2(m), ahead);
        // every thread has read this row's slot
        if (first && row + p.slots < b && *abort == 0) fetch(row + p.slots, this_slot);
        s1 = sums.y;
        k_next = k_after;
        if (!BWD) {
            if (!p.next) continue;
            const float kr = 1.0f / sqrtf(sums.x * inv_h + p.eps);
            if (first && keep && p.rstd_next) p.rstd_next[row] = kr;
            uint8_t *xo = static_cast<uint8_t *>(p.out1) + static_cast<int64_t>(row) * p.H * 2;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = me + j * size;
                if (v >= nvec) continue;
                f2 f[4];
                widen(gn[j], f);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = mul2(mul2(keep_q[j][i], splat(kr)), f[i]);
                if (keep) store8<false>(xo, v, f);
            }
        } else {
            const f2 c2 = splat(p.post ? -k_post * k_post * (sums.x * inv_h) : 0.0f);
            // Without that norm the gradient holds no y, and a zero of c2 alone would make NaN
            // of its infinities and NaN.  (A choice between two results instead of the zeros
            // costs 7 us of 145, 16384 rows of 4096.)
            if (!p.post)
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    if (YF)
#pragma unroll
                        for (int i = 0; i < 4; ++i) yf[YF ? j : 0][i] = 0;
                    else
                        yq[YF ? 0 : j] = make_uint4(0u, 0u, 0u, 0u);
                }
            uint8_t *yo = static_cast<uint8_t *>(p.out1) + static_cast<int64_t>(row) * p.H * (YF ? 4 : 2);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = me + j * size;
                if (v >= nvec) continue;
                f2 y[4];
                if (YF) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = yf[YF ? j : 0][i];
                } else {
                    widen(yq[YF ? 0 : j], y);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = fma2(y[i], c2, keep_q[j][i]);
                if (keep && p.out1) store8<YF>(yo, v, y);
            }
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
    for (int i = first; i < n; i += 8 * step) {      // eight loads at a time
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = i + k * step < n ? __ldg(part + (slot0 + i + k * step) * H + col) : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k & 3] += v[k];
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}
__global__ void __launch_bounds__(32 * RED_WARPS) norm_sums_kernel(const SumParams p) {
    __shared__ float s_red[RED_WARPS][RED_WARPS][33];   // [sequence][warp][column]
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
    // what the warps left in s_red[i], the first warps' sums first
    auto add_warps = [&](int i) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < RED_WARPS; ++w) s += s_red[i][w][lane];
        return s;
    };
    if (blockIdx.y == 0) {
        if (!p.d_gamma_next) return;
        s_red[0][warp][lane] = add_slots(p.part_n, 0, p.nteams, warp, RED_WARPS, p.H, col);
        __syncthreads();
        if (warp == 0 && in) p.d_gamma_next[h] = add_warps(0);
        return;
    }
    if (!p.d_gamma_post && !p.d_gate) return;
    // the teams that have rows of [a, b): team i owns rows [i T / n, (i + 1) T / n)
    auto team_of = [&](int row) {
        int i = static_cast<int>((static_cast<int64_t>(row) * p.nteams) / p.T);
        while (static_cast<int64_t>(i + 1) * p.T / p.nteams <= row) ++i;
        while (static_cast<int64_t>(i) * p.T / p.nteams > row) --i;
        return i;
    };
    auto part_of = [&](int s, int first, int step) {
        const int a = p.seq ? __ldg(p.seq + s) : 0, b = p.seq ? __ldg(p.seq + s + 1) : p.T;
        if (a >= b) return 0.0f;
        const int t0 = team_of(a), t1 = team_of(b - 1);
        return add_slots(p.part_c, static_cast<int64_t>(t0) + s, t1 - t0 + 1, first, step, p.H, col);
    };
    const float gp = bf(p.gamma_post, col);
    float gamma = 0.0f;
    if (p.S < RED_WARPS) {
        for (int s = 0; s < p.S; ++s) s_red[s][warp][lane] = part_of(s, warp, RED_WARPS);
        __syncthreads();
        float c = 0.0f;
        if (warp < p.S) {
            c = add_warps(warp);
            if (p.d_gate && in) p.d_gate[static_cast<int64_t>(warp) * p.H + h] = gp * c;
            gamma = bf(p.gate, static_cast<int64_t>(warp) * p.H + col) * c;
        }
        __syncthreads();
    } else {
        for (int s = warp; s < p.S; s += RED_WARPS) {
            const float c = part_of(s, 0, 1);
            if (p.d_gate && in) p.d_gate[static_cast<int64_t>(s) * p.H + h] = gp * c;
            gamma = fmaf(bf(p.gate, static_cast<int64_t>(s) * p.H + col), c, gamma);
        }
    }
    if (p.d_gamma_post) {
        s_red[0][warp][lane] = gamma;
        __syncthreads();
        if (warp == 0 && in) p.d_gamma_post[h] = add_warps(0);
    }
}

// ------------------------------------------------------------------ host side
inline bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename K, typename P>
cudaError_t start(K kernel, dim3 grid, int block, int smem, const P &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
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
    const dim3 grid(static_cast<unsigned>(ceil_div(p.nteams, sh.teams)));
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
    // rows in the ring: as many as two CTAs a multiprocessor have room for, or one
    // where that is less than two (a row and the next one are needed at once)
    const int row = sh.teams * at;
    p.slots = std::min(MAX_SLOTS, 104 * 1024 / row);
    if (p.slots < 2) p.slots = std::min(MAX_SLOTS, MAX_SMEM / row);
    if (p.slots < 2) return cudaErrorInvalidValue;
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
    if (start(norm_sums_kernel, dim3(static_cast<unsigned>(ceil_div(H, 32)), 2), 32 * RED_WARPS, 0, q, s) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}
