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
    int B, T, D, form, scale, cblocks;
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

// One CTA walks the tiles of one sequence and 32 V channels in order.
template <int V, typename Tx, typename Tg>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Args p) {
    __shared__ float sA[2][kWarps][32 * V], sH[2][kWarps][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / p.cblocks, c = (blockIdx.x % p.cblocks) * 32 * V + lane * V;
    const bool on = c < p.D;
    const int len = length_of(p, b);
    const bool want_b = p.scale != kNone;
    const Tx* x = static_cast<const Tx*>(p.x) + b * p.xb + c;
    const Tg* gate = static_cast<const Tg*>(p.gate) + b * p.gb + c;
    Tx* h = p.h ? static_cast<Tx*>(p.h) + b * p.hb + c : nullptr;
    const int tiles = (len + kTile - 1) / kTile, all_tiles = (p.T + kTile - 1) / kTile;

    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = 0.f;
    if (on && p.h0) load_vec<V>(p.h0 + (int64_t)b * p.D + c, carry);

    for (int tile = 0; tile < tiles; ++tile) {
        const int t0 = tile * kTile + warp * kRun, par = tile & 1;
        float P[kRun][V], H[kRun][V];
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const bool in = on && t0 + j < len;
            float xv[V], gv[V];
            if (in) {
                load_vec<V>(x + (t0 + j) * p.xt, xv);
                load_vec<V>(gate + (t0 + j) * p.gt, gv);
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
        store_vec<V>(&sA[par][warp][lane * V], P[kRun - 1]);
        store_vec<V>(&sH[par][warp][lane * V], H[kRun - 1]);
        __syncthreads();
        float hin[V];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp)
#pragma unroll
                for (int v = 0; v < V; ++v) hin[v] = carry[v];
            float A[V], E[V];
            load_vec<V>(&sA[par][w][lane * V], A);
            load_vec<V>(&sH[par][w][lane * V], E);
#pragma unroll
            for (int v = 0; v < V; ++v) carry[v] = fmaf(A[v], carry[v], E[v]);
        }
        if (on && p.ckpt && warp == 0) store_vec<V>(p.ckpt + ((int64_t)b * all_tiles + tile) * p.D + c, hin);
        if (on && h) {
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
    if (on && p.final_h && warp == 0) store_vec<V>(p.final_h + (int64_t)b * p.D + c, carry);
}

// One CTA walks the tiles of one sequence and 32 V channels from the last to the first; the states
// h_{t-1} are run again from the state that the forward saved at the tile's start.
template <int V, typename Tx, typename Tg>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const Args p) {
    __shared__ float sA[2][kWarps][32 * V], sH[2][kWarps][32 * V], sM[2][kWarps][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / p.cblocks, c = (blockIdx.x % p.cblocks) * 32 * V + lane * V;
    const bool on = c < p.D;
    const int len = length_of(p, b);
    const bool want_b = p.scale != kNone;
    const Tx* x = static_cast<const Tx*>(p.x) + b * p.xb + c;
    const Tg* gate = static_cast<const Tg*>(p.gate) + b * p.gb + c;
    const Tx* dh = static_cast<const Tx*>(p.dh) + b * p.hb + c;
    Tx* dx = static_cast<Tx*>(p.dx) + (int64_t)b * p.T * p.D + c;
    Tg* dgate = static_cast<Tg*>(p.dgate) + (int64_t)b * p.T * p.D + c;
    const int tiles = (len + kTile - 1) / kTile, all_tiles = (p.T + kTile - 1) / kTile;

    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = 0.f;
    if (on && p.dfinal) load_vec<V>(p.dfinal + (int64_t)b * p.D + c, carry);

    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int t0 = tile * kTile + warp * kRun, par = tile & 1;
        float a[kRun][V], bb[kRun][V], xv[kRun][V], dv[kRun][V], hin[V];
#pragma unroll
        for (int v = 0; v < V; ++v) hin[v] = 0.f;
        if (on) load_vec<V>(p.ckpt_in + ((int64_t)b * all_tiles + tile) * p.D + c, hin);
        float A[V], E[V], M[V];
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, E[v] = M[v] = 0.f;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const bool in = on && t0 + j < len;
            float gv[V];
            if (in) {
                load_vec<V>(x + (t0 + j) * p.xt, xv[j]);
                load_vec<V>(gate + (t0 + j) * p.gt, gv);
                load_vec<V>(dh + (t0 + j) * p.ht, dv[j]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (in) {
                    float ds;
                    decay_of(gv[v], p.form, want_b, a[j][v], bb[j][v]);
                    E[v] = fmaf(a[j][v], E[v], scale_of(a[j][v], bb[j][v], p.scale, ds) * xv[j][v]);
                } else {
                    a[j][v] = 1.f;
                    bb[j][v] = xv[j][v] = dv[j][v] = 0.f;
                }
                A[v] *= a[j][v];
            }
        }
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) M[v] = a[j][v] * (dv[j][v] + M[v]);
        store_vec<V>(&sA[par][warp][lane * V], A);
        store_vec<V>(&sH[par][warp][lane * V], E);
        store_vec<V>(&sM[par][warp][lane * V], M);
        __syncthreads();
        float mu[V];
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            if (w == warp)
#pragma unroll
                for (int v = 0; v < V; ++v) mu[v] = carry[v];
            load_vec<V>(&sA[par][w][lane * V], A);
            load_vec<V>(&sM[par][w][lane * V], M);
#pragma unroll
            for (int v = 0; v < V; ++v) carry[v] = fmaf(A[v], carry[v], M[v]);
        }
        for (int w = 0; w < warp; ++w) {
            load_vec<V>(&sA[par][w][lane * V], A);
            load_vec<V>(&sH[par][w][lane * V], E);
#pragma unroll
            for (int v = 0; v < V; ++v) hin[v] = fmaf(A[v], hin[v], E[v]);
        }
        float before[kRun][V];   // h_{t-1}
#pragma unroll
        for (int j = 0; j < kRun; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float ds;
                before[j][v] = hin[v];
                hin[v] = fmaf(a[j][v], hin[v], scale_of(a[j][v], bb[j][v], p.scale, ds) * xv[j][v]);
            }
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) {
            float ox[V], og[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float ds;
                const float lam = dv[j][v] + mu[v];
                const float s = scale_of(a[j][v], bb[j][v], p.scale, ds);
                ox[v] = s * lam;
                og[v] = lam * slope_of(a[j][v], bb[j][v], p.form) * fmaf(xv[j][v], ds, before[j][v]);
                mu[v] = a[j][v] * lam;
            }
            if (on && t0 + j < len) {
                store_vec<V>(dx + (int64_t)(t0 + j) * p.D, ox);
                store_vec<V>(dgate + (int64_t)(t0 + j) * p.D, og);
            }
        }
    }
    if (on && p.dh0 && warp == 0) store_vec<V>(p.dh0 + (int64_t)b * p.D + c, carry);
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
