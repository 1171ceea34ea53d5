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
#include "common.cuh"

namespace osdn {
namespace recur {

enum GateForm : int { kDecay = 0, kLog = 1, kLogit = 2 };      // a = g, exp(g), 1 / (1 + exp(-g))
enum InputScale : int { kNone = 0, kComplement = 1, kNorm = 2 };  // s = 1, 1 - a, sqrt(1 - a^2)

constexpr int kWarps = 8;               // runs of one tile
constexpr int kRun = 8;                 // tokens of one run, held in registers
constexpr int kTile = kWarps * kRun;    // 64: also the distance of the saved states
constexpr int kThreads = 32 * kWarps;

// a and b = 1 - a (b without the cancellation of 1 - a where a is a function of the gate).
__device__ __forceinline__ void decay_of(float g, int form, bool want_b, float& a, float& b) {
    if (form == kDecay) {
        a = g;
        b = 1.f - g;
    } else if (form == kLog) {
        a = expf(g);
        b = want_b ? -expm1f(g) : 0.f;
    } else {
        const float e = expf(-fabsf(g)), r = __fdividef(1.f, 1.f + e), er = e * r;
        a = g >= 0.f ? r : er;
        b = g >= 0.f ? er : r;
    }
}

// s, and ds/da (0 where s = 0: the slope of the root is unbounded there).
__device__ __forceinline__ float scale_of(float a, float b, int scale, float& ds) {
    if (scale == kNone) {
        ds = 0.f;
        return 1.f;
    }
    if (scale == kComplement) {
        ds = -1.f;
        return b;
    }
    const float y = b * (1.f + a);
    const float r = y > 0.f ? rsqrtf(y) : 0.f;
    ds = -a * r;
    return y * r;
}

__device__ __forceinline__ float slope_of(float a, float b, int form) {   // da / dgate
    return form == kDecay ? 1.f : form == kLog ? a : a * b;
}

struct Args {
    const void *x, *gate, *dh;
    const float *h0, *ckpt_in, *dfinal;
    const int* lengths;
    void *h, *dx, *dgate;
    float *final_h, *ckpt, *dh0;
    int B, T, D, form, scale, cblocks, R;
    int64_t xb, xt, gb, gt, hb, ht;     // element strides of x, gate and h (or dh) over (b, t)
};

template <int V, typename T> __device__ __forceinline__ void load_vec(const T* p, float* o) {
    if constexpr (V == 1) o[0] = to_f32(*p);
    else VecIO<V, T>::load(p, o);
}
template <int V, typename T> __device__ __forceinline__ void store_vec(T* p, const float* o) {
    if constexpr (V == 1) *p = from_f32<T>(o[0]);
    else VecIO<V, T>::store(p, o);
}

__device__ __forceinline__ int length_of(const Args& p, int b) {
    if (!p.lengths) return p.T;
    const int n = p.lengths[b];
    return n < 0 ? 0 : n > p.T ? p.T : n;
}

// ---- tiles in shared memory

template <typename T> constexpr int kTileBytes(int V) { return kTile * 32 * V * (int)sizeof(T); }

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool read) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Starts the copy of tokens t0 .. t0 + 63 of 32 V channels (channel c0 on) into tile [64][32 V]; tokens
// from len on and channels from D on are zeros and not read. All threads, 16 bytes each at a time.
template <int V, typename T>
__device__ __forceinline__ void fetch_tile(T* tile, const T* base, int64_t stride, int t0, int len, int c0, int D) {
    constexpr int kPer = 16 / sizeof(T), kRow = 32 * V / kPer;   // elements of 16 bytes, such pieces of a row
#pragma unroll
    for (int i = 0; i < kTile * kRow / kThreads; ++i) {
        const int k = threadIdx.x + i * kThreads, row = k / kRow, col = (k % kRow) * kPer;
        const bool in = t0 + row < len && c0 + col < D;
        cp_async16(tile + row * 32 * V + col, in ? base + (int64_t)(t0 + row) * stride + col : base, in);
    }
}

// ---- joining the CTAs of a cluster

__device__ __forceinline__ void store_remote(float2* local, int rank, float2 v) {
    uint32_t a = (uint32_t)__cvta_generic_to_shared(local), r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(r), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The incoming value of each run of a tile, by one thread a channel. part[w] = (product, end from 0) of
// run w, carry = the value before the cluster's tiles; the runs and the CTAs are taken in the order
// of the walk (kUp: first to last). Writes in[w], returns through `entry` the value before this CTA's tile and
// updates carry to the value behind all of the cluster's tiles.
template <int V, bool kUp>
__device__ __forceinline__ void join_runs(const float* partA, const float* partE, float* in, float2 (*slots)[32 * V],
                                          int R, int rank, float& carry, float& entry) {
    const int ch = threadIdx.x;
    float A[kWarps], E[kWarps], a = 1.f, e = 0.f;
    if (ch < 32 * V) {
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const int w = kUp ? i : kWarps - 1 - i;
            A[i] = partA[w * 32 * V + ch];
            E[i] = partE[w * 32 * V + ch];
            e = fmaf(A[i], e, E[i]);
            a *= A[i];
        }
        for (int r = 0; R > 1 && r < R; ++r) store_remote(&slots[rank][ch], r, make_float2(a, e));
    }
    if (R > 1) cluster_sync();
    if (ch < 32 * V) {
        entry = carry;
        if (R > 1) {
            for (int i = 0; i < R; ++i) {
                const int r = kUp ? i : R - 1 - i;
                const float2 s = slots[r][ch];
                if (r == rank) entry = carry;
                carry = fmaf(s.x, carry, s.y);
            }
        } else {
            carry = fmaf(a, carry, e);
        }
        float v = entry;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            in[(kUp ? i : kWarps - 1 - i) * 32 * V + ch] = v;
            v = fmaf(A[i], v, E[i]);
        }
    }
}

constexpr int kStages = 3;              // tiles in flight or in use
constexpr int kMaxCluster = 16;

// Dynamic shared memory: the stages, then the cluster's slots [2][R][32 V] (none for one CTA).
template <int V, bool kAsync, typename Tx, typename Tg> constexpr int fwd_slots() {
    return kAsync ? kStages * (kTileBytes<Tx>(V) + kTileBytes<Tg>(V)) : 0;
}
template <int V, bool kAsync, typename Tx, typename Tg> constexpr int bwd_slots() {
    return kAsync ? kStages * (2 * kTileBytes<Tx>(V) + kTileBytes<Tg>(V)) : 0;
}
template <int V> constexpr int slot_bytes(int R) { return R > 1 ? 2 * R * 32 * V * (int)sizeof(float2) : 0; }

// A cluster of R CTAs walks one sequence and 32 V channels, R tiles at a time.
template <int V, bool kAsync, typename Tx, typename Tg>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Args p) {
    constexpr int W = 32 * V;
    extern __shared__ __align__(16) char dyn[];
    Tx* bx = reinterpret_cast<Tx*>(dyn);                                        // [kStages][kTile][W]
    Tg* bg = reinterpret_cast<Tg*>(dyn + kStages * kTileBytes<Tx>(V));
    __shared__ float sA[kWarps][W], sE[kWarps][W], sIn[kWarps][W];
    auto slots = reinterpret_cast<float2(*)[W]>(dyn + fwd_slots<V, kAsync, Tx, Tg>());   // [2][R][W]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.R, rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int b = unit / p.cblocks, c0 = (unit % p.cblocks) * W, c = c0 + lane * V;
    const bool on = c < p.D;
    const int len = length_of(p, b);
    const bool want_b = p.scale != kNone;
    const Tx* x = static_cast<const Tx*>(p.x) + b * p.xb + c0;
    const Tg* gate = static_cast<const Tg*>(p.gate) + b * p.gb + c0;
    Tx* h = p.h ? static_cast<Tx*>(p.h) + b * p.hb + c : nullptr;
    const int tiles = (len + kTile - 1) / kTile, all_tiles = (p.T + kTile - 1) / kTile;
    const int steps = (tiles + R - 1) / R;

    const int ch = threadIdx.x;                     // channel whose runs this thread joins
    const bool joins = ch < W && c0 + ch < p.D;
    float carry = joins && p.h0 ? p.h0[(int64_t)b * p.D + c0 + ch] : 0.f, entry = 0.f;

    auto fetch = [&](int i) {
        if (kAsync && i < steps) {
            const int t0 = (i * R + rank) * kTile;
            fetch_tile<V>(bx + (i % kStages) * kTile * W, x, p.xt, t0, len, c0, p.D);
            fetch_tile<V>(bg + (i % kStages) * kTile * W, gate, p.gt, t0, len, c0, p.D);
        }
        if (kAsync) cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    if (kAsync) cp_async_wait<kStages - 2>();
    __syncthreads();

    for (int i = 0; i < steps; ++i) {
        const int t0 = (i * R + rank) * kTile + warp * kRun;
        float P[kRun][V], H[kRun][V];
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const bool in = on && t0 + j < len;
            float xv[V], gv[V];
            if (kAsync) {
                const int at = ((i % kStages) * kTile + warp * kRun + j) * W + lane * V;
                load_vec<V>(bx + at, xv);
                load_vec<V>(bg + at, gv);
            } else if (in) {
                load_vec<V>(x + lane * V + (t0 + j) * p.xt, xv);
                load_vec<V>(gate + lane * V + (t0 + j) * p.gt, gv);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a = 1.f, bb, ds, u = 0.f;
                if (in) {
                    decay_of(gv[v], p.form, want_b, a, bb);
                    u = scale_of(a, bb, p.scale, ds) * xv[v];
                }
                P[j][v] = j ? a * P[j ? j - 1 : 0][v] : a;
                H[j][v] = j ? fmaf(a, H[j ? j - 1 : 0][v], u) : u;
            }
        }
        store_vec<V>(&sA[warp][lane * V], P[kRun - 1]);
        store_vec<V>(&sE[warp][lane * V], H[kRun - 1]);
        __syncthreads();
        fetch(i + kStages - 1);
        join_runs<V, true>(&sA[0][0], &sE[0][0], &sIn[0][0], slots + (i & 1) * R, R, rank, carry, entry);
        if (joins && p.ckpt && i * R + rank < tiles)
            p.ckpt[((int64_t)b * all_tiles + i * R + rank) * p.D + c0 + ch] = entry;
        if (kAsync) cp_async_wait<kStages - 2>();
        __syncthreads();
        if (on && h) {
            float hin[V];
            load_vec<V>(&sIn[warp][lane * V], hin);
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (t0 + j < len) {
                    float o[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] = fmaf(P[j][v], hin[v], H[j][v]);
                    store_vec<V>(h + (t0 + j) * p.ht, o);
                }
        }
    }
    if (joins && p.final_h && rank == 0) p.final_h[(int64_t)b * p.D + c0 + ch] = carry;
}

// A cluster of R CTAs walks the tiles of one sequence and 32 V channels from the last to the first; the
// states h_{t-1} are run again from the state that the forward saved at the tile's start.
template <int V, bool kAsync, typename Tx, typename Tg>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const Args p) {
    constexpr int W = 32 * V;
    extern __shared__ __align__(16) char dyn[];
    Tx* bx = reinterpret_cast<Tx*>(dyn);                                        // [kStages][kTile][W]
    Tx* bd = reinterpret_cast<Tx*>(dyn + kStages * kTileBytes<Tx>(V));
    Tg* bg = reinterpret_cast<Tg*>(dyn + 2 * kStages * kTileBytes<Tx>(V));
    __shared__ float sA[kWarps][W], sE[kWarps][W], sM[kWarps][W], sH[kWarps][W], sIn[kWarps][W];
    auto slots = reinterpret_cast<float2(*)[W]>(dyn + bwd_slots<V, kAsync, Tx, Tg>());   // [2][R][W]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.R, rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int b = unit / p.cblocks, c0 = (unit % p.cblocks) * W, c = c0 + lane * V;
    const bool on = c < p.D;
    const int len = length_of(p, b);
    const bool want_b = p.scale != kNone;
    const Tx* x = static_cast<const Tx*>(p.x) + b * p.xb + c0;
    const Tg* gate = static_cast<const Tg*>(p.gate) + b * p.gb + c0;
    const Tx* dh = static_cast<const Tx*>(p.dh) + b * p.hb + c0;
    Tx* dx = static_cast<Tx*>(p.dx) + (int64_t)b * p.T * p.D + c;
    Tg* dgate = static_cast<Tg*>(p.dgate) + (int64_t)b * p.T * p.D + c;
    const int tiles = (len + kTile - 1) / kTile, all_tiles = (p.T + kTile - 1) / kTile;
    const int steps = (tiles + R - 1) / R;

    const int ch = threadIdx.x;
    const bool joins = ch < W && c0 + ch < p.D;
    float carry = joins && p.dfinal ? p.dfinal[(int64_t)b * p.D + c0 + ch] : 0.f, entry = 0.f;
    auto tile_of = [&](int i) { return (steps - 1 - i) * R + rank; };

    auto fetch = [&](int i) {
        if (kAsync && i < steps) {
            const int t0 = tile_of(i) * kTile, s = (i % kStages) * kTile * W;
            fetch_tile<V>(bx + s, x, p.xt, t0, len, c0, p.D);
            fetch_tile<V>(bg + s, gate, p.gt, t0, len, c0, p.D);
            fetch_tile<V>(bd + s, dh, p.ht, t0, len, c0, p.D);
        }
        if (kAsync) cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    if (kAsync) cp_async_wait<kStages - 2>();
    __syncthreads();

    for (int i = 0; i < steps; ++i) {
        const int tile = tile_of(i), t0 = tile * kTile + warp * kRun;
        const int at0 = ((i % kStages) * kTile + warp * kRun) * W + lane * V;
        float start = joins && tile < tiles ? p.ckpt_in[((int64_t)b * all_tiles + tile) * p.D + c0 + ch] : 0.f;
        float a[kRun][V], bb[kRun][V], xr[kAsync ? 1 : kRun][V], dr[kAsync ? 1 : kRun][V];
        auto x_at = [&](int j, float* o) {          // x and dh of token j: again from the tile, or kept
            if constexpr (kAsync) load_vec<V>(bx + at0 + j * W, o);
            else
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = xr[j][v];
        };
        auto dh_at = [&](int j, float* o) {
            if constexpr (kAsync) load_vec<V>(bd + at0 + j * W, o);
            else
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = dr[j][v];
        };
        float A[V], E[V], M[V];
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, E[v] = M[v] = 0.f;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const bool in = on && t0 + j < len;
            float xv[V], gv[V];
            if constexpr (kAsync) {
                load_vec<V>(bg + at0 + j * W, gv);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) gv[v] = xr[j][v] = dr[j][v] = 0.f;
                if (in) {
                    load_vec<V>(x + lane * V + (t0 + j) * p.xt, xr[j]);
                    load_vec<V>(gate + lane * V + (t0 + j) * p.gt, gv);
                    load_vec<V>(dh + lane * V + (t0 + j) * p.ht, dr[j]);
                }
            }
            x_at(j, xv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                a[j][v] = 1.f;
                bb[j][v] = 0.f;
                if (in) {
                    float ds;
                    decay_of(gv[v], p.form, want_b, a[j][v], bb[j][v]);
                    E[v] = fmaf(a[j][v], E[v], scale_of(a[j][v], bb[j][v], p.scale, ds) * xv[v]);
                }
                A[v] *= a[j][v];
            }
        }
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) {
            float dv[V];
            dh_at(j, dv);                            // zeros behind the length
#pragma unroll
            for (int v = 0; v < V; ++v) M[v] = a[j][v] * (dv[v] + M[v]);
        }
        store_vec<V>(&sA[warp][lane * V], A);
        store_vec<V>(&sE[warp][lane * V], E);
        store_vec<V>(&sM[warp][lane * V], M);
        __syncthreads();
        fetch(i + kStages - 1);
        if (ch < W) {                                // the states before each run
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                sH[w][ch] = start;
                start = fmaf(sA[w][ch], start, sE[w][ch]);
            }
        }
        join_runs<V, false>(&sA[0][0], &sM[0][0], &sIn[0][0], slots + (i & 1) * R, R, rank, carry, entry);
        if (kAsync) cp_async_wait<kStages - 2>();
        __syncthreads();
        float hin[V], mu[V];
        load_vec<V>(&sH[warp][lane * V], hin);
        load_vec<V>(&sIn[warp][lane * V], mu);
        float before[kRun][V];                       // h_{t-1}
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            float xv[V];
            x_at(j, xv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float ds;
                before[j][v] = hin[v];
                hin[v] = fmaf(a[j][v], hin[v], scale_of(a[j][v], bb[j][v], p.scale, ds) * xv[v]);
            }
        }
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) {
            float ox[V], og[V], xv[V], dv[V];
            x_at(j, xv);
            dh_at(j, dv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float ds;
                const float lam = dv[v] + mu[v];
                const float s = scale_of(a[j][v], bb[j][v], p.scale, ds);
                ox[v] = s * lam;
                og[v] = lam * slope_of(a[j][v], bb[j][v], p.form) * fmaf(xv[v], ds, before[j][v]);
                mu[v] = a[j][v] * lam;
            }
            if (on && t0 + j < len) {
                store_vec<V>(dx + (int64_t)(t0 + j) * p.D, ox);
                store_vec<V>(dgate + (int64_t)(t0 + j) * p.D, og);
            }
        }
    }
    if (joins && p.dh0 && rank == 0) p.dh0[(int64_t)b * p.D + c0 + ch] = carry;
}

// One token for every channel: state <- a state + s x in place, h = the new state.
template <int V, typename Tx, typename Tg>
__global__ void __launch_bounds__(256) step_kernel(const Args p) {
    const int per = p.D / V;
    const int64_t n = (int64_t)p.B * per;
    const bool want_b = p.scale != kNone;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t b = i / per, c = (i - b * per) * V;
        float xv[V], gv[V], st[V];
        load_vec<V>(static_cast<const Tx*>(p.x) + b * p.xb + c, xv);
        load_vec<V>(static_cast<const Tg*>(p.gate) + b * p.gb + c, gv);
        load_vec<V>(p.final_h + b * p.D + c, st);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a, bb, ds;
            decay_of(gv[v], p.form, want_b, a, bb);
            st[v] = fmaf(a, st[v], scale_of(a, bb, p.scale, ds) * xv[v]);
        }
        store_vec<V>(p.final_h + b * p.D + c, st);
        store_vec<V>(static_cast<Tx*>(p.h) + b * p.hb + c, st);
    }
}

}  // namespace recur
}  // namespace osdn
