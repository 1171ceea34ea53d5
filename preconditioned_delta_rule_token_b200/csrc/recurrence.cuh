// Gated linear recurrence over the tokens of every channel, its backward and its single-token step.
//
// With a_t and s_t made from the gate (GateForm, InputScale):
//   h_t = a_t h_{t-1} + s_t x_t                                  (forward, h_0 given)
//   lam_t = dh_t + mu_{t+1},  mu_t = a_t lam_t,  mu_{N+1} = dh_N (backward; dh_0 = mu_1)
//   dx_t = s_t lam_t,  dgate_t = lam_t a'_t (h_{t-1} + x_t ds/da)
// A run of tokens maps its incoming state affinely, h_out = A h_in + H with A the product of its
// a_t and H its end state from 0, and mu_out = A mu_in + M the other way. So a CTA takes a tile of
// kTile tokens x 32 V channels, each warp runs its kRun tokens from 0, and the runs are joined
// through shared memory in the order of the tokens.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace osdn {
namespace recur {

enum GateForm : int { kDecay = 0, kLog = 1, kLogit = 2 };      // a = g, exp(g), 1 / (1 + exp(-g))
enum InputScale : int { kNone = 0, kComplement = 1, kNorm = 2 };  // s = 1, 1 - a, sqrt(1 - a^2)

constexpr int kSaved = 64;              // tokens between the saved states
constexpr int kWarps = 8;               // runs of one tile, a warp each
constexpr int kThreads = 32 * kWarps;
// Tokens of one run, held in registers (forward, backward). More of them join fewer runs.
template <bool kTma, typename Tx, typename Tg> constexpr int fwd_run() {
    return !kTma || sizeof(Tx) + sizeof(Tg) > 6 ? 8 : 16;
}
constexpr int kBwdRun = 8;

// ---- two channels at a time: one instruction for both where sm_100a has it (fma, mul, add on f32x2)

__device__ __forceinline__ uint64_t bits2(float2 a) { return *reinterpret_cast<uint64_t*>(&a); }
__device__ __forceinline__ float2 pair2(uint64_t a) { return *reinterpret_cast<float2*>(&a); }
__device__ __forceinline__ float2 all2(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return pair2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 less1(float2 a) { return fma2(a, all2(-1.f), all2(1.f)); }   // 1 - a

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float root(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rroot(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// a and b = 1 - a, each without the cancellation of taking it from the other where that one is near 1:
// a product of thousands of decays near 1 shows any bias of a single one.
//   log:   |g| < 0.2: b = -g q(g) with q the polynomial of degree 4 that meets (e^g - 1) / g at the
//          Chebyshev points of that range (within 3e-8 of it), a = 1 - b; else a = 2^(g log2 e), b = 1 - a;
//   logit: with e = exp(-|g|) and m = e / (1 + e) <= 1/2, a and b are m and 1 - m by the sign of g.
template <int kForm> __device__ __forceinline__ void decay_of(float2 g, float2& a, float2& b) {
    constexpr float kLog2e = 1.4426950408889634f;
    if constexpr (kForm == kDecay) {
        a = g;
        b = less1(g);
    } else if constexpr (kForm == kLog) {
        const float2 t = mul2(g, all2(kLog2e));
        const float2 la = make_float2(ex2(t.x), ex2(t.y));
        const float2 lb = less1(la);
        float2 s = fma2(g, all2(-0.00834326f), all2(-0.041736159f));
        s = fma2(g, s, all2(-0.16666657f));
        s = fma2(g, s, all2(-0.49999931f));
        s = fma2(g, s, all2(-1.f));
        const float2 sb = mul2(g, s), sa = less1(sb);
        const bool x = fabsf(g.x) < 0.2f, y = fabsf(g.y) < 0.2f;
        a = make_float2(x ? sa.x : la.x, y ? sa.y : la.y);
        b = make_float2(x ? sb.x : lb.x, y ? sb.y : lb.y);
    } else {
        const float2 e = make_float2(ex2(-kLog2e * fabsf(g.x)), ex2(-kLog2e * fabsf(g.y)));
        const float2 d = add2(e, all2(1.f));
        const float2 m = mul2(e, make_float2(rcp(d.x), rcp(d.y)));
        const float2 q = less1(m);
        a = make_float2(g.x >= 0.f ? q.x : m.x, g.y >= 0.f ? q.y : m.y);
        b = make_float2(g.x >= 0.f ? m.x : q.x, g.y >= 0.f ? m.y : q.y);
    }
}

template <int kScale> __device__ __forceinline__ float2 scale_of(float2 a, float2 b) {
    if constexpr (kScale == kNone) return all2(1.f);
    if constexpr (kScale == kComplement) return b;
    const float2 y = fma2(a, b, b);
    return make_float2(root(y.x), root(y.y));
}

// s, and ds/da (0 where s = 0: the slope of the root is unbounded there).
template <int kScale> __device__ __forceinline__ float2 scale_of(float2 a, float2 b, float2& ds) {
    if constexpr (kScale == kNone) {
        ds = all2(0.f);
        return all2(1.f);
    }
    if constexpr (kScale == kComplement) {
        ds = all2(-1.f);
        return b;
    }
    const float2 y = fma2(a, b, b);
    const float2 r = make_float2(y.x > 0.f ? rroot(y.x) : 0.f, y.y > 0.f ? rroot(y.y) : 0.f);
    ds = mul2(a, mul2(r, all2(-1.f)));
    return mul2(y, r);
}

template <int kForm> __device__ __forceinline__ float2 slope_of(float2 a, float2 b) {   // da / dgate
    if constexpr (kForm == kDecay) return all2(1.f);
    if constexpr (kForm == kLog) return a;
    return mul2(a, b);
}

// f(form, scale) as constants: one branch for all that a thread does with them.
template <typename F> __device__ __forceinline__ void with_kind(int form, int scale, F&& f) {
    auto scales = [&](auto fo) {
        if (scale == kNone) f(fo, std::integral_constant<int, kNone>{});
        else if (scale == kComplement) f(fo, std::integral_constant<int, kComplement>{});
        else f(fo, std::integral_constant<int, kNorm>{});
    };
    if (form == kDecay) scales(std::integral_constant<int, kDecay>{});
    else if (form == kLog) scales(std::integral_constant<int, kLog>{});
    else scales(std::integral_constant<int, kLogit>{});
}

struct Args {
    const void *x, *gate, *dh;
    const float *h0, *ckpt_in, *dfinal;
    const int* lengths;
    void *h, *dx, *dgate;
    float *final_h, *ckpt, *dh0;
    int B, T, D, form, scale, cblocks, R;
    unsigned long long wait_limit_ns;
    int64_t xb, xt, gb, gt, hb, ht;     // element strides of x, gate and h (or dh) over (b, t)
};

// V (1 or 2) channels as a pair; the second of one channel is 0 and not stored.
template <int V, typename T> __device__ __forceinline__ float2 load_pair(const T* p) {
    if constexpr (V == 1) {
        return make_float2(to_f32(*p), 0.f);
    } else if constexpr (sizeof(T) == 2) {          // bf16 is the upper half of fp32
        const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
        return *reinterpret_cast<const float2*>(p);
    }
}
template <int V, typename T> __device__ __forceinline__ void store_pair(T* p, float2 v) {
    if constexpr (V == 1) {
        *p = from_f32<T>(v.x);
    } else {
        const float o[2] = {v.x, v.y};
        VecIO<2, T>::store(p, o);
    }
}

__device__ __forceinline__ int length_of(const Args& p, int b) {
    if (!p.lengths) return p.T;
    const int n = p.lengths[b];
    return n < 0 ? 0 : n > p.T ? p.T : n;
}

// ---- tiles in shared memory, by the tensor memory accelerator

constexpr int kMaxCluster = 16;

template <typename T> constexpr int kTileBytes(int V, int run) { return kWarps * run * 32 * V * (int)sizeof(T); }

// Tensor maps over [B, T, D] (innermost first: channels, tokens, sequences): loads of a tile, stores of a run.
struct Maps {
    CUtensorMap x, gate, dh;            // loads
    CUtensorMap o0, o1;                 // stores: h, or dx and dgate
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c, int t, int b, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(t), "r"(b), "r"(tc::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c, int t, int b) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(tc::smem_u32(src)), "r"(c), "r"(t), "r"(b)
                 : "memory");
}

// The stages' barriers: one phase a use, waited for by every thread. A wait that passes the limit
// sets the library's status word; later waits of that thread are then skipped, so the kernel still ends.
template <int kStages> struct Pipe {
    uint64_t* full;                     // [kStages]
    unsigned long long limit_ns;
    bool failed;
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
        if (!failed && !tc::mbar_wait(bar, parity, limit_ns)) {
            failed = true;
            atomicOr(&g_osdn_status, kStatusTimeout);
        }
    }
    __device__ __forceinline__ void wait(int i) { wait(full + i % kStages, (i / kStages) & 1); }
    // Copies that were started and not waited for, before the block leaves (only after a failed wait).
    __device__ __forceinline__ void drain(int from, int to) {
        if (!failed) return;
        for (int i = from; i < to; ++i) tc::mbar_wait(full + i % kStages, (i / kStages) & 1, 1000000000ull);
    }
};

// ---- joining the CTAs of a cluster

__device__ __forceinline__ uint32_t at_rank(const void* local, int rank) {   // the same address in CTA `rank`
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(local)), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What the CTAs of a cluster tell one another each step: (product, end from 0) of their tile for a lane's two
// channels, stored into every CTA's slots with the bytes counted on that CTA's barrier, so a step needs no
// fence. Two sets by the step's parity: a CTA sends for step i + 2 after all its warps have had step i + 1 from
// every CTA, and those sent that after their warps had read step i.
struct Exchange {
    float4 (*slots)[32];                // [2][R]
    uint64_t* bar;                      // [2]
    int R, rank;
    __device__ __forceinline__ void init() {
        if (R == 1) return;
        if (threadIdx.x == 0) {
            tc::mbar_init(bar, 1);
            tc::mbar_init(bar + 1, 1);
            tc::fence_mbar_init();
        }
        cluster_sync();
    }
    __device__ __forceinline__ void send(int i, int lane, float2 a, float2 e) {   // one warp of the CTA
        if (lane == 0) tc::mbar_arrive_expect_tx(bar + (i & 1), R * 32 * (int)sizeof(float4));
        const float4* slot = &slots[(i & 1) * R + rank][lane];
        for (int r = 0; r < R; ++r)
            asm volatile(
                "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                    at_rank(slot, r)),
                "f"(a.x), "f"(a.y), "f"(e.x), "f"(e.y), "r"(at_rank(bar + (i & 1), r))
                : "memory");
    }
};

// The value that comes into this warp's run. A[w], E[w] = (product, end from 0) of run w for the lane's
// channels; carry = the value before the cluster's tiles, the same in every warp and CTA. Runs and CTAs are
// taken in the order of the walk (kUp: first to last). entry = the value before this CTA's tile; carry
// becomes the value behind all of the cluster's tiles.
template <int V, bool kUp, typename P>
__device__ __forceinline__ float2 join_runs(const float (*A)[32 * V], const float (*E)[32 * V], Exchange& ex, P& pipe,
                                            int i, float2& carry, float2& entry) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2 in = carry;
    entry = carry;
    if (ex.R == 1) {
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const int w = kUp ? k : kWarps - 1 - k;
            if (w == warp) in = carry;
            carry = fma2(load_pair<V>(&A[w][lane * V]), carry, load_pair<V>(&E[w][lane * V]));
        }
        return in;
    }
    float2 a = all2(1.f), e = all2(0.f), pa = a, pe = e;
    const bool sends = warp == (i & (kWarps - 1));   // in turn
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        const int w = kUp ? k : kWarps - 1 - k;
        if (w == warp) {
            pa = a;
            pe = e;
            if (!sends) break;
        }
        const float2 aw = load_pair<V>(&A[w][lane * V]);
        e = fma2(aw, e, load_pair<V>(&E[w][lane * V]));
        a = mul2(a, aw);
    }
    if (sends) ex.send(i, lane, a, e);
    pipe.wait(ex.bar + (i & 1), (i >> 1) & 1);
    for (int k = 0; k < ex.R; ++k) {
        const int r = kUp ? k : ex.R - 1 - k;
        const float4 s = ex.slots[(i & 1) * ex.R + r][lane];
        if (r == ex.rank) entry = carry;
        carry = fma2(make_float2(s.x, s.y), carry, make_float2(s.z, s.w));
    }
    return fma2(pa, entry, pe);
}

// Dynamic shared memory: the stages (128-byte aligned), then the cluster's slots [2][R][32] (none for one CTA).
template <typename Tx, typename Tg> constexpr int fwd_stages() { return sizeof(Tx) + sizeof(Tg) == 6 ? 2 : 3; }
constexpr int kBwdStages = 3;
template <int V, bool kTma, typename Tx, typename Tg> constexpr int fwd_slots() {
    constexpr int run = fwd_run<kTma, Tx, Tg>();
    return kTma ? fwd_stages<Tx, Tg>() * (kTileBytes<Tx>(V, run) + kTileBytes<Tg>(V, run)) : 0;
}
template <int V, bool kTma, typename Tx, typename Tg> constexpr int bwd_slots() {
    return kTma ? kBwdStages * (2 * kTileBytes<Tx>(V, kBwdRun) + kTileBytes<Tg>(V, kBwdRun)) : 0;
}
constexpr int kSlotBytes = 2 * 32 * (int)sizeof(float4);   // each CTA's

// A cluster of R CTAs walks one sequence and 32 V channels, R tiles at a time.
template <int V, bool kTma, typename Tx, typename Tg>
__global__ void __launch_bounds__(kThreads, 2) fwd_kernel(const Args p, const __grid_constant__ Maps maps) {
    constexpr int W = 32 * V, kRun = fwd_run<kTma, Tx, Tg>(), kStages = fwd_stages<Tx, Tg>(), kTile = kWarps * kRun;
    extern __shared__ __align__(128) char dyn[];
    Tx* bx = reinterpret_cast<Tx*>(dyn);                                        // [kStages][kTile][W]
    Tg* bg = reinterpret_cast<Tg*>(dyn + kStages * kTileBytes<Tx>(V, kRun));
    auto slots = reinterpret_cast<float4(*)[32]>(dyn + fwd_slots<V, kTma, Tx, Tg>());   // [2][R]
    __shared__ float sA[2][kWarps][W], sE[2][kWarps][W];   // by the step's parity
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.R, rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int b = unit / p.cblocks, c0 = (unit % p.cblocks) * W, c = c0 + lane * V;
    const bool on = c < p.D;
    const int len = length_of(p, b);
    const Tx* x = static_cast<const Tx*>(p.x) + b * p.xb + c0;
    const Tg* gate = static_cast<const Tg*>(p.gate) + b * p.gb + c0;
    Tx* h = p.h ? static_cast<Tx*>(p.h) + b * p.hb + c : nullptr;
    const int tiles = (len + kTile - 1) / kTile, saved = (p.T + kSaved - 1) / kSaved;
    const int steps = (tiles + R - 1) / R;

    float2 carry = all2(0.f), entry;
    if (on && p.h0) carry = load_pair<V>(p.h0 + (int64_t)b * p.D + c);

    __shared__ uint64_t full[kStages];
    Pipe<kStages> pipe{full, p.wait_limit_ns, false};
    __shared__ uint64_t joined[2];
    Exchange ex{slots, joined, R, rank};
    ex.init();
    auto fetch = [&](int i) {                       // starts the copies of this CTA's i-th tile (thread 0)
        if (kTma && threadIdx.x == 0 && i < steps) {
            const int t0 = (i * R + rank) * kTile, s = i % kStages;
            tc::mbar_arrive_expect_tx(full + s, kTileBytes<Tx>(V, kRun) + kTileBytes<Tg>(V, kRun));
            tma_load_3d(bx + s * kTile * W, &maps.x, c0, t0, b, full + s);
            tma_load_3d(bg + s * kTile * W, &maps.gate, c0, t0, b, full + s);
        }
    };
    if (kTma) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < kStages; ++s) tc::mbar_init(full + s, 1);
            tc::fence_mbar_init();
        }
        __syncthreads();
        for (int i = 0; i < kStages - 1; ++i) fetch(i);
    }

    for (int i = 0; i < steps; ++i) {
        const int t0 = (i * R + rank) * kTile + warp * kRun;
        const int live = kTma || on ? len - t0 : 0;   // tokens of this run inside the sequence
        float2 P[kRun], H[kRun];
        if (kTma) pipe.wait(i);
        const int at0 = ((i % kStages) * kTile + warp * kRun) * W + lane * V;
        with_kind(p.form, p.scale, [&](auto form, auto scale) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                float2 xv = all2(0.f), gv = all2(0.f), a, bb;
                if constexpr (kTma) {
                    xv = load_pair<V>(bx + at0 + j * W);
                    gv = load_pair<V>(bg + at0 + j * W);
                } else if (j < live) {
                    xv = load_pair<V>(x + lane * V + (t0 + j) * p.xt);
                    gv = load_pair<V>(gate + lane * V + (t0 + j) * p.gt);
                }
                decay_of<form>(gv, a, bb);
                H[j] = scale == kNone ? xv : mul2(scale_of<scale>(a, bb), xv);
                P[j] = a;
            }
        });
        if (live < kRun) {                          // tokens behind the length change nothing
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (j >= live) P[j] = all2(1.f), H[j] = all2(0.f);
        }
#pragma unroll
        for (int j = 1; j < kRun; ++j) {
            H[j] = fma2(P[j], H[j - 1], H[j]);
            P[j] = mul2(P[j], P[j - 1]);
        }
        store_pair<V>(&sA[i & 1][warp][lane * V], P[kRun - 1]);
        store_pair<V>(&sE[i & 1][warp][lane * V], H[kRun - 1]);
        if (kTma && lane == 0) tc::bulk_wait_read<0>();   // the last tile has left: its stage is free
        __syncthreads();
        fetch(i + kStages - 1);
        const float2 hin = join_runs<V, true>(sA[i & 1], sE[i & 1], ex, pipe, i, carry, entry);
        if (warp % (kSaved / kRun) == 0 && on && p.ckpt && t0 < len)
            store_pair<V>(p.ckpt + ((int64_t)b * saved + t0 / kSaved) * p.D + c, hin);
        if (kTma && h && live >= kRun) {            // a whole run: over its own x in the tile, and out from there
#pragma unroll
            for (int j = 0; j < kRun; ++j) store_pair<V>(bx + at0 + j * W, fma2(P[j], hin, H[j]));
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(&maps.o0, bx + at0, c0, t0, b);
                tc::bulk_commit();
            }
        } else if (h && on && live > 0) {
            Tx* o = h + t0 * p.ht;
            if (live >= kRun) {
#pragma unroll
                for (int j = 0; j < kRun; ++j, o += p.ht) store_pair<V>(o, fma2(P[j], hin, H[j]));
            } else {
#pragma unroll
                for (int j = 0; j < kRun; ++j, o += p.ht)
                    if (j < live) store_pair<V>(o, fma2(P[j], hin, H[j]));
            }
        }
    }
    if (warp == 0 && on && p.final_h && rank == 0) store_pair<V>(p.final_h + (int64_t)b * p.D + c, carry);
    if (kTma) {
        pipe.drain(0, steps);
        if (lane == 0) tc::bulk_wait_read<0>();
    }
    if (R > 1) cluster_sync();   // no CTA leaves while another may still store to it
}

// A cluster of R CTAs walks the tiles of one sequence and 32 V channels from the last to the first; the
// states h_{t-1} are run again from the state that the forward saved at the tile's start.
template <int V, bool kTma, typename Tx, typename Tg>
__global__ void __launch_bounds__(kThreads, 2) bwd_kernel(const Args p, const __grid_constant__ Maps maps) {
    constexpr int W = 32 * V, kRun = kBwdRun, kStages = kBwdStages, kTile = kWarps * kRun;
    extern __shared__ __align__(128) char dyn[];
    Tx* bx = reinterpret_cast<Tx*>(dyn);                                        // [kStages][kTile][W]
    Tx* bd = reinterpret_cast<Tx*>(dyn + kStages * kTileBytes<Tx>(V, kRun));
    Tg* bg = reinterpret_cast<Tg*>(dyn + 2 * kStages * kTileBytes<Tx>(V, kRun));
    auto slots = reinterpret_cast<float4(*)[32]>(dyn + bwd_slots<V, kTma, Tx, Tg>());   // [2][R]
    __shared__ float sA[2][kWarps][W], sE[2][kWarps][W], sM[2][kWarps][W];   // by the step's parity
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.R, rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int b = unit / p.cblocks, c0 = (unit % p.cblocks) * W, c = c0 + lane * V;
    const bool on = c < p.D;
    const int len = length_of(p, b);
    const Tx* x = static_cast<const Tx*>(p.x) + b * p.xb + c0;
    const Tg* gate = static_cast<const Tg*>(p.gate) + b * p.gb + c0;
    const Tx* dh = static_cast<const Tx*>(p.dh) + b * p.hb + c0;
    Tx* dx = static_cast<Tx*>(p.dx) + (int64_t)b * p.T * p.D + c;
    Tg* dgate = static_cast<Tg*>(p.dgate) + (int64_t)b * p.T * p.D + c;
    const int tiles = (len + kTile - 1) / kTile, all_tiles = (p.T + kTile - 1) / kTile;
    static_assert(kTile == kSaved, "a saved state before each tile");
    const int steps = (tiles + R - 1) / R;

    float2 carry = all2(0.f), entry;
    if (on && p.dfinal) carry = load_pair<V>(p.dfinal + (int64_t)b * p.D + c);
    auto tile_of = [&](int i) { return (steps - 1 - i) * R + rank; };

    __shared__ uint64_t full[kStages];
    Pipe<kStages> pipe{full, p.wait_limit_ns, false};
    __shared__ uint64_t joined[2];
    Exchange ex{slots, joined, R, rank};
    ex.init();
    auto fetch = [&](int i) {
        if (kTma && threadIdx.x == 0 && i < steps) {
            const int t0 = tile_of(i) * kTile, s = i % kStages;
            tc::mbar_arrive_expect_tx(full + s, 2 * kTileBytes<Tx>(V, kRun) + kTileBytes<Tg>(V, kRun));
            tma_load_3d(bx + s * kTile * W, &maps.x, c0, t0, b, full + s);
            tma_load_3d(bg + s * kTile * W, &maps.gate, c0, t0, b, full + s);
            tma_load_3d(bd + s * kTile * W, &maps.dh, c0, t0, b, full + s);
        }
    };
    if (kTma) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < kStages; ++s) tc::mbar_init(full + s, 1);
            tc::fence_mbar_init();
        }
        __syncthreads();
        for (int i = 0; i < kStages - 1; ++i) fetch(i);
    }

    auto saved = [&](int i) {                        // the state before the CTA's i-th tile
        const int tile = tile_of(i);
        return on && i < steps && tile < tiles
                   ? load_pair<V>(p.ckpt_in + ((int64_t)b * all_tiles + tile) * p.D + c)
                   : all2(0.f);
    };
    float2 next = saved(0);
    for (int i = 0; i < steps; ++i) {
        const int t0 = tile_of(i) * kTile + warp * kRun;
        const int live = kTma || on ? len - t0 : 0;
        const int at0 = ((i % kStages) * kTile + warp * kRun) * W + lane * V;
        float2 state = next;                         // before the tile, then before this run
        float2 a[kRun], bb[kRun], xr[kTma ? 1 : kRun] = {}, dr[kTma ? 1 : kRun] = {};
        auto x_at = [&](int j) {                     // x and dh of token j: again from the tile, or kept
            if constexpr (kTma) return load_pair<V>(bx + at0 + j * W);
            else return xr[j];
        };
        auto dh_at = [&](int j) {
            if constexpr (kTma) return load_pair<V>(bd + at0 + j * W);
            else return dr[j];
        };
        float2 A = all2(1.f), E = all2(0.f), M = all2(0.f);
        if (kTma) {
            pipe.wait(i);
            if (live < kRun) {                       // whatever lies behind the length counts as zeros
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (j >= live) {
                        store_pair<V>(bx + at0 + j * W, all2(0.f));
                        store_pair<V>(bd + at0 + j * W, all2(0.f));
                        store_pair<V>(bg + at0 + j * W, all2(0.f));
                    }
            }
        }
        with_kind(p.form, p.scale, [&](auto form, auto scale) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                float2 gv = all2(0.f);
                if constexpr (kTma) {
                    gv = load_pair<V>(bg + at0 + j * W);
                } else if (j < live) {
                    xr[j] = load_pair<V>(x + lane * V + (t0 + j) * p.xt);
                    gv = load_pair<V>(gate + lane * V + (t0 + j) * p.gt);
                    dr[j] = load_pair<V>(dh + lane * V + (t0 + j) * p.ht);
                }
                decay_of<form>(gv, a[j], bb[j]);
                if (!kTma && j >= live) a[j] = all2(1.f);
            }
            if (kTma && live < kRun) {
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (j >= live) a[j] = all2(1.f);
            }
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const float2 xv = x_at(j);
                E = fma2(a[j], E, scale == kNone ? xv : mul2(scale_of<scale>(a[j], bb[j]), xv));
                A = mul2(A, a[j]);
            }
        });
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) M = mul2(a[j], add2(dh_at(j), M));
        store_pair<V>(&sA[i & 1][warp][lane * V], A);
        store_pair<V>(&sE[i & 1][warp][lane * V], E);
        store_pair<V>(&sM[i & 1][warp][lane * V], M);
        if (kTma && lane == 0) tc::bulk_wait_read<0>();
        __syncthreads();
        fetch(i + kStages - 1);
        next = saved(i + 1);
        float2 mu = join_runs<V, false>(sA[i & 1], sM[i & 1], ex, pipe, i, carry, entry);
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
            if (w < warp) state = fma2(load_pair<V>(&sA[i & 1][w][lane * V]), state, load_pair<V>(&sE[i & 1][w][lane * V]));
        if (live > 0) {
            float2 lam[kRun];
#pragma unroll
            for (int j = kRun - 1; j >= 0; --j) {
                lam[j] = add2(dh_at(j), mu);
                mu = mul2(a[j], lam[j]);
            }
            Tx* ox = dx + (int64_t)t0 * p.D;
            Tg* og = dgate + (int64_t)t0 * p.D;
            with_kind(p.form, p.scale, [&](auto form, auto scale) {
#pragma unroll
                for (int j = 0; j < kRun; ++j, ox += p.D, og += p.D) {
                    float2 ds;
                    const float2 xv = x_at(j), s = scale_of<scale>(a[j], bb[j], ds);
                    float2 g = scale == kNone ? state : fma2(xv, ds, state);   // state: h_{t-1}
                    g = mul2(form == kDecay ? lam[j] : mul2(lam[j], slope_of<form>(a[j], bb[j])), g);
                    state = fma2(a[j], state, scale == kNone ? xv : mul2(s, xv));
                    const float2 d = scale == kNone ? lam[j] : mul2(s, lam[j]);
                    if (kTma) {                      // over their own tiles, and out from there
                        store_pair<V>(bx + at0 + j * W, d);
                        store_pair<V>(bg + at0 + j * W, g);
                    } else if (j < live) {
                        store_pair<V>(ox, d);
                        store_pair<V>(og, g);
                    }
                }
            });
            if (kTma && live >= kRun) {
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&maps.o0, bx + at0, c0, t0, b);
                    tma_store_3d(&maps.o1, bg + at0, c0, t0, b);
                    tc::bulk_commit();
                }
            } else if (kTma && on) {
                ox = dx + (int64_t)t0 * p.D;
                og = dgate + (int64_t)t0 * p.D;
                for (int j = 0; j < live; ++j, ox += p.D, og += p.D) {
                    store_pair<V>(ox, load_pair<V>(bx + at0 + j * W));
                    store_pair<V>(og, load_pair<V>(bg + at0 + j * W));
                }
            }
        }
    }
    if (warp == 0 && on && p.dh0 && rank == 0) store_pair<V>(p.dh0 + (int64_t)b * p.D + c, carry);
    if (kTma) {
        pipe.drain(0, steps);
        if (lane == 0) tc::bulk_wait_read<0>();
    }
    if (R > 1) cluster_sync();   // no CTA leaves while another may still store to it
}

// One token for every channel: state <- a state + s x in place, h = the new state.
template <int V, typename Tx, typename Tg>
__global__ void __launch_bounds__(256) step_kernel(const Args p) {
    constexpr int kPairs = V == 4 ? 2 : 1;
    const int per = p.D / V;
    const int64_t n = (int64_t)p.B * per;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t b = i / per, c = (i - b * per) * V;
        float xv[4] = {}, gv[4] = {}, st[4] = {};
        if constexpr (V == 4) {
            VecIO<4, Tx>::load(static_cast<const Tx*>(p.x) + b * p.xb + c, xv);
            VecIO<4, Tg>::load(static_cast<const Tg*>(p.gate) + b * p.gb + c, gv);
            VecIO<4, float>::load(p.final_h + b * p.D + c, st);
        } else {
            xv[0] = to_f32(static_cast<const Tx*>(p.x)[b * p.xb + c]);
            gv[0] = to_f32(static_cast<const Tg*>(p.gate)[b * p.gb + c]);
            st[0] = p.final_h[b * p.D + c];
        }
        with_kind(p.form, p.scale, [&](auto form, auto scale) {
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                float2 a, bb;
                decay_of<form>(make_float2(gv[2 * k], gv[2 * k + 1]), a, bb);
                const float2 u = mul2(scale_of<scale>(a, bb), make_float2(xv[2 * k], xv[2 * k + 1]));
                const float2 r = fma2(a, make_float2(st[2 * k], st[2 * k + 1]), u);
                st[2 * k] = r.x;
                st[2 * k + 1] = r.y;
            }
        });
        if constexpr (V == 4) {
            VecIO<4, float>::store(p.final_h + b * p.D + c, st);
            VecIO<4, Tx>::store(static_cast<Tx*>(p.h) + b * p.hb + c, st);
        } else {
            p.final_h[b * p.D + c] = st[0];
            static_cast<Tx*>(p.h)[b * p.hb + c] = from_f32<Tx>(st[0]);
        }
    }
}

}  // namespace recur
}  // namespace osdn
