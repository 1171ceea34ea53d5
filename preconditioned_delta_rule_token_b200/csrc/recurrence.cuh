// Gated linear recurrence over the tokens of every channel, its backward and its single-token step.
//
// With a_t and s_t made from the gate (GateForm, InputScale):
//   h_t = a_t h_{t-1} + s_t x_t                                  (forward, h_0 given)
//   lam_t = dh_t + mu_{t+1},  mu_t = a_t lam_t,  mu_{N+1} = dh_N (backward; dh_0 = mu_1)
//   dx_t = s_t lam_t,  dgate_t = lam_t a'_t (h_{t-1} + x_t ds/da)
// A run of tokens maps its incoming state affinely, h_out = A h_in + H with A the product of its
// a_t and H its end state from 0, and mu_out = A mu_in + M the other way. So a CTA takes a tile of 8
// runs x 64 channels, each warp goes through its run from 0 with two channels a lane, the runs are joined
// through shared memory in the order of the tokens, and the run's results follow from what comes in.
//
// Why so. The operator reads and writes 6 bytes an element forward and 10 backward (bf16) for 10 to 40
// operations, so memory bounds it; but a walk over the tokens is serial, and 148 SMs need more of them at a
// time than there are channels / 64. A cluster of R CTAs therefore takes R tiles at a time and exchanges one
// pair a channel through distributed shared memory: no second pass over the data, no flag in device
// memory, and the same result on every run. R is the most (up to 16) at which all clusters are resident.
// Measured on the way (bf16 forward, B8 T4096 D2048, log gate, norm scale / B1 T32768, fp32 log gate):
// one CTA a walk with plain loads 648 / 3720 us; clusters with a hardware barrier each step 255 / 242;
// packed arithmetic 114 / 165; tensor-map tiles and counted remote stores 107 / 108; 16 tokens a run instead
// of 8 in the forward (half the joins) 83 / 95; unpacking bf16 by shifts 79 / 92 us, 79% and 90% of
// the measured copy rate. The second is bound by memory. The first puts 256 equal CTAs on 296 places: the 108 SMs
// that hold two set the time and issue 2.6 of 4 a cycle (21 instructions an element), the 40 that hold one are
// done after two thirds of it; over all SMs 2.2 of 4 and 4.4 TB/s. The backward, B8 T4096 D2048:
// 141 us (logit, complement), 156 us (log, norm), 74% and 67%: 44 instructions an element in two walks over a
// run, and two CTAs an SM by registers. What did not pay in the forward: 16 warps a CTA (111 us where 8 took
// 102), two warps that join for all behind a second barrier (107), scalar arithmetic (34 instructions, 105).
// Rows that are not whole 16 bytes, B8 T2048 D1001 against D1024 with the same bytes an element: fp32 forward 67
// us against 35, with the backward 169 against 95; bf16 84 against 25, and 187 against 72 (kLoads has none ahead).
#pragma once
#include <type_traits>

#include "pairs.cuh"
#include "tc_ptx.cuh"

namespace osdn {
namespace recur {

enum GateForm : int { kDecay = 0, kLog = 1, kLogit = 2 };      // a = g, exp(g), 1 / (1 + exp(-g))
enum InputScale : int { kNone = 0, kComplement = 1, kNorm = 2 };  // s = 1, 1 - a, sqrt(1 - a^2)

constexpr int kSaved = 64;              // tokens between the saved states
constexpr int kWarps = 8;               // runs of one tile, a warp each
constexpr int kThreads = 32 * kWarps;
constexpr int W = 64;                   // channels of one tile, two a lane
// Tokens of one run, held in registers (forward, backward): 16 halve the joins against 8 (107 -> 83 us at B8
// T4096 D2048 bf16); fp32 tiles of 16 would leave one CTA to an SM, and the backward's arrays do not fit.
template <typename Tx, typename Tg> constexpr int fwd_run() { return sizeof(Tx) + sizeof(Tg) > 6 ? 8 : 16; }
constexpr int kBwdRun = 8;

// ---- the gate

constexpr float kLeast = 1.17549435e-38f;   // the least normal number

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

// s, and ds/da (0 where s = 0: the slope of the root is unbounded there). The root and its reciprocal take a
// 1 - a^2 below the normal range as 0, which the reciprocal would make infinite: s = 0 there, as forward.
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
    const float2 r = make_float2(y.x >= kLeast ? rroot(y.x) : 0.f, y.y >= kLeast ? rroot(y.y) : 0.f);
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
    int B, T, D, form, scale, cblocks, R, zero_rest;
    unsigned long long wait_limit_ns;
    int64_t xb, xt, gb, gt, hb, ht;     // element strides of x, gate and h (or dh) over (b, t)
};

// Two neighbouring channels, from and to addresses on whole pairs (bf16 is the upper half of fp32).
__device__ __forceinline__ float2 load_pair(const __nv_bfloat16* p) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 load_pair(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float2 v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ void store_pair(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }

// A lane's two channels in device memory, kStep apart: 1, from and to whole pairs, or 32, where rows may start
// anywhere and a warp still reads and writes whole runs of them. n: how many of the two are inside the row.
template <int kStep, typename T> __device__ __forceinline__ float2 get_pair(const T* p, int n) {
    if constexpr (kStep == 1) return n ? load_pair(p) : all2(0.f);
    else return make_float2(n > 0 ? to_f32(p[0]) : 0.f, n > 1 ? to_f32(p[kStep]) : 0.f);
}
template <int kStep, typename T> __device__ __forceinline__ void put_pair(T* p, float2 v, int n) {
    if constexpr (kStep == 1) {
        if (n) store_pair(p, v);
    } else {
        if (n > 0) p[0] = from_f32<T>(v.x);
        if (n > 1) p[kStep] = from_f32<T>(v.y);
    }
}

__device__ __forceinline__ int length_of(const Args& p, int b) {
    if (!p.lengths) return p.T;
    const int n = p.lengths[b];
    return n < 0 ? 0 : n > p.T ? p.T : n;
}

// ---- tiles in shared memory

// How tokens come into the tiles: kTma, by tensor maps, a thread a tile (rows and widths in whole 16 bytes);
// kCopies, each thread its own pairs by asynchronous copies of 4 bytes (fp32, or bf16 on whole pairs);
// kLoads, its own pairs by plain loads, without any ahead (bf16 rows that start inside a pair).
enum Mode : int { kTma = 0, kCopies = 1, kLoads = 2 };
template <int kMode, typename Tx> constexpr int channel_step() {
    return kMode == kLoads || (kMode == kCopies && sizeof(Tx) == 4) ? 32 : 1;
}
constexpr int kMaxCluster = 16;

template <typename T> constexpr int kTileBytes(int run) { return kWarps * run * W * (int)sizeof(T); }

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

__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool read) {   // 4 zero bytes if not read
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(read ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One thread's pair of kRun tokens into its place in the tile (rows W apart), the first `live` of them and n
// channels; the rest are zeros and not read (their copies of no bytes name `any`, the tensor's start).
template <int kMode, int kRun, int kStep, typename T>
__device__ __forceinline__ void fetch_own(T* own, const T* row, int64_t stride, int live, int n, const T* any) {
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        const int m = j < live ? n : 0;
        const T* src = m ? row + j * stride : any;
        if constexpr (kMode == kLoads) {
            own[j * W] = m > 0 ? src[0] : from_f32<T>(0.f);
            own[j * W + 1] = m > 1 ? src[kStep] : from_f32<T>(0.f);
        } else if constexpr (sizeof(T) == 2) {
            cp_async4(own + j * W, src, m > 0);
        } else {
            cp_async4(own + j * W, src, m > 0);
            cp_async4(own + j * W + 1, m > 1 ? src + kStep : any, m > 1);
        }
    }
}

// The stages' barriers: one phase a use, waited for by every thread. A wait that passes the limit sets the
// library's status word; that thread then waits and sends no more, so that the kernel still ends (its
// results are undefined), and the thread that starts the copies lets those in flight land first.
template <int kStages> struct Pipe {
    uint64_t* full;                     // [kStages]
    unsigned long long limit_ns;
    bool failed;
    int started;                        // tiles whose copies this thread has started
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
        if (failed) return;
        // a try suspends the thread for some microseconds; under a shorter limit the phase is only looked at
        auto ready = [&] { return limit_ns < 20000ull ? tc::mbar_test(bar, parity) : tc::mbar_try_wait(bar, parity); };
        if (ready()) return;
        const uint64_t t0 = tc::globaltimer_ns();
        while (!ready())
            if (tc::globaltimer_ns() - t0 > limit_ns) {
                failed = true;
                atomicOr(&g_osdn_status, kStatusTimeout);
                return;
            }
    }
    __device__ __forceinline__ void wait(int i) { wait(full + i % kStages, (i / kStages) & 1); }
    // Before the block leaves, only after a failed wait: copies into its tiles, and a cluster's stores (100 us).
    __device__ __forceinline__ void drain(int R) {
        if (!failed) return;
        for (int i = max(0, started - kStages); i < started; ++i)
            tc::mbar_wait(full + i % kStages, (i / kStages) & 1, 1000000000ull);
        if (R > 1)
            for (const uint64_t t0 = tc::globaltimer_ns(); tc::globaltimer_ns() - t0 < 100000;) {}
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
template <bool kUp, typename P>
__device__ __forceinline__ float2 join_runs(const float (*A)[W], const float (*E)[W], Exchange& ex, P& pipe,
                                            int i, float2& carry, float2& entry) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2 in = carry;
    entry = carry;
    if (ex.R == 1) {
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const int w = kUp ? k : kWarps - 1 - k;
            if (w == warp) in = carry;
            carry = fma2(load_pair(&A[w][lane * 2]), carry, load_pair(&E[w][lane * 2]));
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
        const float2 aw = load_pair(&A[w][lane * 2]);
        e = fma2(aw, e, load_pair(&E[w][lane * 2]));
        a = mul2(a, aw);
    }
    if (sends && !pipe.failed) ex.send(i, lane, a, e);
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
// Three tiles in flight or in use (two: 97 us instead of 83 at B8 T4096 D2048 bf16); two where three would leave
// one CTA to an SM (fp32 gates at B1 T32768: three 120 us, two 95 us).
template <typename Tx, typename Tg> constexpr int fwd_stages() { return sizeof(Tx) + sizeof(Tg) == 6 ? 2 : 3; }
// Backward: three, two with fp32 gates, where three CTAs to an SM then pay for the registers that they spill
// (B1 T16384 D2048: 98 us against 128; with bf16 gates they cost, B8 T4096 D2048 156 us against 141).
template <typename Tx, typename Tg> constexpr int bwd_stages() { return sizeof(Tg) == 4 ? 2 : 3; }
template <typename Tx, typename Tg> constexpr int fwd_slots() {
    constexpr int run = fwd_run<Tx, Tg>();
    return fwd_stages<Tx, Tg>() * (kTileBytes<Tx>(run) + kTileBytes<Tg>(run));
}
template <typename Tx, typename Tg> constexpr int bwd_slots() {
    return bwd_stages<Tx, Tg>() * (2 * kTileBytes<Tx>(kBwdRun) + kTileBytes<Tg>(kBwdRun));
}
constexpr int kSlotBytes = 2 * 32 * (int)sizeof(float4);   // each CTA's

// A cluster of R CTAs walks one sequence and 64 channels, R tiles at a time.
template <int kMode, typename Tx, typename Tg>
__global__ void __launch_bounds__(kThreads, 2) fwd_kernel(const Args p, const __grid_constant__ Maps maps) {
    constexpr int kRun = fwd_run<Tx, Tg>(), kStages = fwd_stages<Tx, Tg>(), kTile = kWarps * kRun;
    constexpr int kStep = channel_step<kMode, Tx>();
    extern __shared__ __align__(128) char dyn[];
    Tx* bx = reinterpret_cast<Tx*>(dyn);                                        // [kStages][kTile][W]
    Tg* bg = reinterpret_cast<Tg*>(dyn + kStages * kTileBytes<Tx>(kRun));
    auto slots = reinterpret_cast<float4(*)[32]>(dyn + fwd_slots<Tx, Tg>());    // [2][R]
    __shared__ float sA[2][kWarps][W], sE[2][kWarps][W];   // by the step's parity
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.R, rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int b = unit / p.cblocks, c0 = (unit % p.cblocks) * W, c = c0 + lane * (kStep == 1 ? 2 : 1);
    const int n = (c < p.D) + (c + kStep < p.D);    // this lane's channels inside the row
    __shared__ uint64_t full[kStages];
    Pipe<kStages> pipe{full, p.wait_limit_ns, false, 0};
    __shared__ uint64_t joined[2];
    Exchange ex{slots, joined, R, rank};
    let_next_start();
    ex.init();
    wait_for_previous();
    const int len = length_of(p, b);
    const Tx* x = static_cast<const Tx*>(p.x) + b * p.xb + c;
    const Tg* gate = static_cast<const Tg*>(p.gate) + b * p.gb + c;
    Tx* h = p.h ? static_cast<Tx*>(p.h) + b * p.hb + c : nullptr;
    const int tiles = (len + kTile - 1) / kTile, saved = (p.T + kSaved - 1) / kSaved;
    const int steps = (tiles + R - 1) / R;

    float2 carry = all2(0.f), entry;
    if (p.h0) carry = get_pair<kStep>(p.h0 + (int64_t)b * p.D + c, n);

    auto fetch = [&](int i) {                       // starts the copies of this CTA's i-th tile
        const int t0 = (i * R + rank) * kTile, s = i % kStages;
        if constexpr (kMode == kTma) {
            if (threadIdx.x == 0 && i < steps && !pipe.failed) {
                pipe.started = i + 1;
                tc::mbar_arrive_expect_tx(full + s, kTileBytes<Tx>(kRun) + kTileBytes<Tg>(kRun));
                tma_load_3d(bx + s * kTile * W, &maps.x, c0, t0, b, full + s);
                tma_load_3d(bg + s * kTile * W, &maps.gate, c0, t0, b, full + s);
            }
        } else {
            if (i < steps) {
                const int t = t0 + warp * kRun, at = (s * kTile + warp * kRun) * W + lane * 2;
                fetch_own<kMode, kRun, kStep>(bx + at, x + t * p.xt, p.xt, len - t, n, static_cast<const Tx*>(p.x));
                fetch_own<kMode, kRun, kStep>(bg + at, gate + t * p.gt, p.gt, len - t, n, static_cast<const Tg*>(p.gate));
            }
            cp_async_commit();
        }
    };
    if constexpr (kMode == kTma) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < kStages; ++s) tc::mbar_init(full + s, 1);
            tc::fence_mbar_init();
        }
        __syncthreads();
    }
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    for (int i = 0; i < steps; ++i) {
        const int t0 = (i * R + rank) * kTile + warp * kRun;
        const int live = len - t0;                  // tokens of this run inside the sequence
        const int at0 = ((i % kStages) * kTile + warp * kRun) * W + lane * 2;
        float2 P[kRun], H[kRun];
        if constexpr (kMode == kTma) pipe.wait(i);
        else cp_async_wait<kStages - 2>();
        with_kind(p.form, p.scale, [&](auto form, auto scale) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                float2 a, bb;
                const float2 xv = load_pair(bx + at0 + j * W);
                decay_of<form>(load_pair(bg + at0 + j * W), a, bb);
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
        store_pair(&sA[i & 1][warp][lane * 2], P[kRun - 1]);
        store_pair(&sE[i & 1][warp][lane * 2], H[kRun - 1]);
        if (kMode == kTma && lane == 0) tc::bulk_wait_read<0>();   // the last tile has left: its stage is free
        __syncthreads();
        fetch(i + kStages - 1);
        const float2 hin = join_runs<true>(sA[i & 1], sE[i & 1], ex, pipe, i, carry, entry);
        if (warp % (kSaved / kRun) == 0 && p.ckpt && t0 < len)
            put_pair<kStep>(p.ckpt + ((int64_t)b * saved + t0 / kSaved) * p.D + c, hin, n);
        if (h && live > 0) {
            if (kMode == kTma && live >= kRun) {    // a whole run: over its own x in the tile, and out from there
#pragma unroll
                for (int j = 0; j < kRun; ++j) store_pair(bx + at0 + j * W, fma2(P[j], hin, H[j]));
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&maps.o0, bx + at0, c0, t0, b);
                    tc::bulk_commit();
                }
            } else {
                Tx* o = h + t0 * p.ht;
#pragma unroll
                for (int j = 0; j < kRun; ++j, o += p.ht)
                    if (j < live) put_pair<kStep>(o, fma2(P[j], hin, H[j]), n);
            }
        }
    }
    if (h && p.zero_rest)
        for (int t = len + rank * kWarps + warp; t < p.T; t += R * kWarps) put_pair<kStep>(h + t * p.ht, all2(0.f), n);
    if (p.ckpt && p.lengths) {   // before tokens behind the length: the state that is left
        const int all = (p.T + kSaved - 1) / kSaved;   // not kept from the start: 79 us with it so, 80 us kept
        for (int k = (len + kSaved - 1) / kSaved + rank * kWarps + warp; k < all; k += R * kWarps)
            put_pair<kStep>(p.ckpt + ((int64_t)b * all + k) * p.D + c, carry, n);
    }
    if (warp == 0 && rank == 0 && p.final_h) put_pair<kStep>(p.final_h + (int64_t)b * p.D + c, carry, n);
    if (kMode == kTma && lane == 0) tc::bulk_wait_read<0>();
    pipe.drain(R);
    __syncwarp();
    if (R > 1) cluster_sync();   // no CTA leaves while another may still store to it
}

// A cluster of R CTAs walks the tiles of one sequence and 64 channels from the last to the first. A run first
// walks back for its lam, then forward through its states h_{t-1}, which start from the state that the
// forward saved at the tile's start, and gives dx and dgate on the way.
template <int kMode, typename Tx, typename Tg>
__global__ void __launch_bounds__(kThreads, kMode == kTma && sizeof(Tg) > sizeof(Tx) ? 3 : 2) bwd_kernel(const Args p, const __grid_constant__ Maps maps) {
    constexpr int kRun = kBwdRun, kStages = bwd_stages<Tx, Tg>(), kTile = kWarps * kRun;
    constexpr int kStep = channel_step<kMode, Tx>();
    static_assert(kTile == kSaved, "a saved state before each tile");
    extern __shared__ __align__(128) char dyn[];
    Tx* bx = reinterpret_cast<Tx*>(dyn);                                        // [kStages][kTile][W]
    Tx* bd = reinterpret_cast<Tx*>(dyn + kStages * kTileBytes<Tx>(kRun));
    Tg* bg = reinterpret_cast<Tg*>(dyn + 2 * kStages * kTileBytes<Tx>(kRun));
    auto slots = reinterpret_cast<float4(*)[32]>(dyn + bwd_slots<Tx, Tg>());    // [2][R]
    __shared__ float sA[2][kWarps][W], sE[2][kWarps][W], sM[2][kWarps][W];   // by the step's parity
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.R, rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int b = unit / p.cblocks, c0 = (unit % p.cblocks) * W, c = c0 + lane * (kStep == 1 ? 2 : 1);
    const int n = (c < p.D) + (c + kStep < p.D);
    __shared__ uint64_t full[kStages];
    Pipe<kStages> pipe{full, p.wait_limit_ns, false, 0};
    __shared__ uint64_t joined[2];
    Exchange ex{slots, joined, R, rank};
    let_next_start();
    ex.init();
    wait_for_previous();
    const int len = length_of(p, b);
    const Tx* x = static_cast<const Tx*>(p.x) + b * p.xb + c;
    const Tg* gate = static_cast<const Tg*>(p.gate) + b * p.gb + c;
    const Tx* dh = static_cast<const Tx*>(p.dh) + b * p.hb + c;
    Tx* dx = static_cast<Tx*>(p.dx) + (int64_t)b * p.T * p.D + c;
    Tg* dgate = static_cast<Tg*>(p.dgate) + (int64_t)b * p.T * p.D + c;
    const int tiles = (len + kTile - 1) / kTile, all_tiles = (p.T + kTile - 1) / kTile;
    const int steps = (tiles + R - 1) / R;

    float2 carry = all2(0.f), entry;
    if (p.dfinal) carry = get_pair<kStep>(p.dfinal + (int64_t)b * p.D + c, n);
    auto tile_of = [&](int i) { return (steps - 1 - i) * R + rank; };

    auto fetch = [&](int i) {
        const int t0 = tile_of(i) * kTile, s = i % kStages;
        if constexpr (kMode == kTma) {
            if (threadIdx.x == 0 && i < steps && !pipe.failed) {
                pipe.started = i + 1;
                tc::mbar_arrive_expect_tx(full + s, 2 * kTileBytes<Tx>(kRun) + kTileBytes<Tg>(kRun));
                tma_load_3d(bx + s * kTile * W, &maps.x, c0, t0, b, full + s);
                tma_load_3d(bg + s * kTile * W, &maps.gate, c0, t0, b, full + s);
                tma_load_3d(bd + s * kTile * W, &maps.dh, c0, t0, b, full + s);
            }
        } else {
            if (i < steps) {
                const int t = t0 + warp * kRun, at = (s * kTile + warp * kRun) * W + lane * 2;
                fetch_own<kMode, kRun, kStep>(bx + at, x + t * p.xt, p.xt, len - t, n, static_cast<const Tx*>(p.x));
                fetch_own<kMode, kRun, kStep>(bg + at, gate + t * p.gt, p.gt, len - t, n, static_cast<const Tg*>(p.gate));
                fetch_own<kMode, kRun, kStep>(bd + at, dh + t * p.ht, p.ht, len - t, n, static_cast<const Tx*>(p.dh));
            }
            cp_async_commit();
        }
    };
    if constexpr (kMode == kTma) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < kStages; ++s) tc::mbar_init(full + s, 1);
            tc::fence_mbar_init();
        }
        __syncthreads();
    }
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    auto saved = [&](int i) {                        // the state before the CTA's i-th tile
        const int tile = tile_of(i);
        if (i >= steps || tile >= tiles) return all2(0.f);
        return get_pair<kStep>(p.ckpt_in + ((int64_t)b * all_tiles + tile) * p.D + c, n);
    };
    float2 next = saved(0);
    for (int i = 0; i < steps; ++i) {
        const int t0 = tile_of(i) * kTile + warp * kRun;
        const int live = len - t0;
        const int at0 = ((i % kStages) * kTile + warp * kRun) * W + lane * 2;
        float2 state = next;                         // before the tile, then before this run
        float2 a[kRun], bb[kRun], A = all2(1.f), E = all2(0.f), M = all2(0.f);
        if constexpr (kMode == kTma) {
            pipe.wait(i);
            if (live < kRun) {                       // whatever lies behind the length counts as zeros
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (j >= live) {
                        store_pair(bx + at0 + j * W, all2(0.f));
                        store_pair(bd + at0 + j * W, all2(0.f));
                        store_pair(bg + at0 + j * W, all2(0.f));
                    }
                tc::fence_proxy_async_smem();
            }
        } else {
            cp_async_wait<kStages - 2>();
        }
        with_kind(p.form, p.scale, [&](auto form, auto scale) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) decay_of<form>(load_pair(bg + at0 + j * W), a[j], bb[j]);
            if (live < kRun) {
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (j >= live) a[j] = all2(1.f);
            }
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const float2 xv = load_pair(bx + at0 + j * W);
                E = fma2(a[j], E, scale == kNone ? xv : mul2(scale_of<scale>(a[j], bb[j]), xv));
                A = mul2(A, a[j]);
            }
        });
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) M = mul2(a[j], add2(load_pair(bd + at0 + j * W), M));
        store_pair(&sA[i & 1][warp][lane * 2], A);
        store_pair(&sE[i & 1][warp][lane * 2], E);
        store_pair(&sM[i & 1][warp][lane * 2], M);
        if (kMode == kTma && lane == 0) tc::bulk_wait_read<0>();
        __syncthreads();
        fetch(i + kStages - 1);
        next = saved(i + 1);
        float2 mu = join_runs<false>(sA[i & 1], sM[i & 1], ex, pipe, i, carry, entry);
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
            if (w < warp) state = fma2(load_pair(&sA[i & 1][w][lane * 2]), state, load_pair(&sE[i & 1][w][lane * 2]));
        if (live > 0) {
            float2 lam[kRun];
#pragma unroll
            for (int j = kRun - 1; j >= 0; --j) {
                lam[j] = add2(load_pair(bd + at0 + j * W), mu);
                mu = mul2(a[j], lam[j]);
            }
            Tx* ox = dx + (int64_t)t0 * p.D;
            Tg* og = dgate + (int64_t)t0 * p.D;
            with_kind(p.form, p.scale, [&](auto form, auto scale) {
#pragma unroll
                for (int j = 0; j < kRun; ++j, ox += p.D, og += p.D) {
                    float2 ds;
                    const float2 xv = load_pair(bx + at0 + j * W), s = scale_of<scale>(a[j], bb[j], ds);
                    float2 g = scale == kNone ? state : fma2(xv, ds, state);   // state: h_{t-1}
                    g = mul2(form == kDecay ? lam[j] : mul2(lam[j], slope_of<form>(a[j], bb[j])), g);
                    state = fma2(a[j], state, scale == kNone ? xv : mul2(s, xv));
                    const float2 d = scale == kNone ? lam[j] : mul2(s, lam[j]);
                    if (kMode == kTma) {             // over their own tiles, and out from there
                        store_pair(bx + at0 + j * W, d);
                        store_pair(bg + at0 + j * W, g);
                    } else if (j < live) {
                        put_pair<kStep>(ox, d, n);
                        put_pair<kStep>(og, g, n);
                    }
                }
            });
            if (kMode == kTma) tc::fence_proxy_async_smem();   // before the stores out, or the stage's next copies in
            if (kMode == kTma && live >= kRun) {
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&maps.o0, bx + at0, c0, t0, b);
                    tma_store_3d(&maps.o1, bg + at0, c0, t0, b);
                    tc::bulk_commit();
                }
            } else if (kMode == kTma) {
                ox = dx + (int64_t)t0 * p.D;
                og = dgate + (int64_t)t0 * p.D;
                for (int j = 0; j < live; ++j, ox += p.D, og += p.D) {
                    put_pair<kStep>(ox, load_pair(bx + at0 + j * W), n);
                    put_pair<kStep>(og, load_pair(bg + at0 + j * W), n);
                }
            }
        }
    }
    if (p.zero_rest)
        for (int t = len + rank * kWarps + warp; t < p.T; t += R * kWarps) {
            put_pair<kStep>(dx + (int64_t)t * p.D, all2(0.f), n);
            put_pair<kStep>(dgate + (int64_t)t * p.D, all2(0.f), n);
        }
    if (warp == 0 && rank == 0 && p.dh0) put_pair<kStep>(p.dh0 + (int64_t)b * p.D + c, carry, n);
    if (kMode == kTma && lane == 0) tc::bulk_wait_read<0>();
    pipe.drain(R);
    __syncwarp();
    if (R > 1) cluster_sync();
}

// One token for every channel: state <- a state + s x in place, h = the new state.
template <int V, typename Tx, typename Tg>
__global__ void __launch_bounds__(256) step_kernel(const Args p) {
    constexpr int kPairs = V == 4 ? 2 : 1;
    const int per = p.D / V;
    let_next_start();
    wait_for_previous();
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
