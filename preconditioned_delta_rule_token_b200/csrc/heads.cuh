// Norms of queries and keys for each head with the position rotation in the same pass, the backward
// of both, and (with the norm off) the rotation alone.
//
// For a row x of one token and head, n = 1 (L2) or its width (RMS):
//   inv = (sum x^2 / n + eps)^(-1/2),  y = scale w inv x,  out = m R(theta) y on the first rot
// features and y on the rest, R turning the pairs (i, i + rot/2) or (2i, 2i+1) by
// theta_i = position * freq_i. Backward, with g = scale (m R(-theta)) dout:
//   dw = sum over rows of g inv x,   dx = inv (g w - x inv^2 / n <g w, x>).
// A row lies in a group of lanes, 8 features a lane; its sums and the partner features of the
// half layout go between the lanes by shuffles.
#pragma once
#include "common.cuh"

namespace osdn {
namespace heads {

enum Norm : int { kNoNorm = 0, kL2 = 1, kRms = 2 };
enum Layout : int { kHalf = 0, kInterleaved = 1 };

constexpr int kThreads = 256;
constexpr int kVec = 8;             // features a lane
constexpr int kMaxWidth = 256;

struct Side {                       // one of q and k
    const void *x, *dout;           // dout: backward only
    void* out;                      // out, or dx in the backward
    const float* w;                 // norm weights or NULL
    float* dw;                      // partial sums of the weights' gradient [grid][width] or NULL
    Tok3 sx, so;                    // strides of x, and of out (forward) or dout (backward)
    Tok3 sd;                        // strides of dx (backward)
    int H;
    float scale;
};

struct Args {
    Side side[2];
    const long long* positions;     // [B, T] or NULL: pos0 + t
    const double* freqs;            // [rot / 2]
    const int* lengths;             // [B] or NULL
    long long pos0, tokens;         // tokens = B * T
    int T, width, rot, norm, layout, inverse;
    float eps, amplitude;
};

template <typename T> __device__ __forceinline__ void load8(const T* p, float* o) {
    VecIO<4, T>::load(p, o);
    VecIO<4, T>::load(p + 4, o + 4);
}
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* o) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float* o) {
    VecIO<4, T>::store(p, o);
    VecIO<4, T>::store(p + 4, o + 4);
}
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float* o) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 a = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&a);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the G lanes of a group (every lane of the warp takes part).
template <int G> __device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// m cos and m sin of position * freq: the angle in turns and its whole turns taken off in 64 bits
// (a far position times a frequency leaves no digits of the angle in 32), the rest in 32.
__device__ __forceinline__ float2 cos_sin(double position, double freq, float amplitude) {
    const double turns = position * freq * 0.15915494309189533577;
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    return make_float2(amplitude * c, amplitude * s);
}

// Rotate the lane's 8 features y (feature e0 of the row on); cs: this token's table; sign -1 turns back.
template <int G>
__device__ __forceinline__ void rotate(float* y, const float2* cs, int gl, int rot, int layout, float sign) {
    const int e0 = gl * kVec;
    if (layout == kInterleaved) {
#pragma unroll
        for (int i = 0; i < kVec; i += 2)
            if (e0 + i < rot) {
                const float2 t = cs[(e0 + i) >> 1];
                const float a = y[i], b = y[i + 1], sn = sign * t.y;
                y[i] = a * t.x - b * sn;
                y[i + 1] = b * t.x + a * sn;
            }
    } else {
        const int half = rot / (2 * kVec);          // lanes of one half
        const bool in = gl < 2 * half, lower = gl < half;
        const int lane = threadIdx.x & 31;
        const int src = !in ? lane : lower ? lane + half : lane - half;
        const float sg = lower ? -sign : sign;
        const int f0 = lower ? e0 : e0 - rot / 2;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const float other = __shfl_sync(0xffffffffu, y[i], src);
            if (in) {
                const float2 t = cs[f0 + i];
                y[i] = y[i] * t.x + other * (sg * t.y);
            }
        }
    }
}

// A CTA takes kTok tokens at a time: their table of cosines, then their rows of q and of k.
template <int G, int kTok, bool kBackward, typename Tx>
__global__ void __launch_bounds__(kThreads) heads_kernel(const Args p) {
    extern __shared__ float2 table[];               // [kTok][rot / 2]
    __shared__ longlong2 where[kTok];               // sequence and token of each; token -1: past a length
    __shared__ float sums[kBackward ? kThreads * kVec : 1];
    constexpr int kGroups = kThreads / G;
    const int group = threadIdx.x / G, gl = threadIdx.x % G, e0 = gl * kVec;
    const bool on = e0 < p.width;
    const int pairs = p.rot / 2;
    const float n_inv = p.norm == kRms ? 1.f / (float)p.width : 1.f;
    float dw[2][kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) dw[0][i] = dw[1][i] = 0.f;

    for (long long tok0 = (long long)blockIdx.x * kTok; tok0 < p.tokens; tok0 += (long long)gridDim.x * kTok) {
        __syncthreads();                            // the previous tokens' table has been read
        if (threadIdx.x < kTok) {
            const long long tok = tok0 + threadIdx.x, b = tok / p.T, t = tok - b * p.T;
            const bool live = tok < p.tokens && (!p.lengths || t < p.lengths[b]);
            where[threadIdx.x] = make_longlong2(b, live ? t : -1);
        }
        for (int i = threadIdx.x; i < kTok * pairs; i += kThreads) {
            const long long tok = tok0 + i / pairs;
            if (tok < p.tokens) {
                const long long pos = p.positions ? p.positions[tok] : p.pos0 + tok % p.T;
                table[i] = cos_sin((double)pos, p.freqs[i % pairs], p.amplitude);
            }
        }
        __syncthreads();
#pragma unroll
        for (int sd = 0; sd < 2; ++sd) {
            const Side& s = p.side[sd];
            const int rows = kTok * s.H;
            float w[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) w[i] = 1.f;
            if (on && s.w) load8<float>(s.w + e0, w);
            for (int r0 = 0; r0 < rows; r0 += kGroups) {   // every lane of a warp takes part in the shuffles
                const int r = r0 + group, k = r / max(s.H, 1), head = r - k * s.H;
                const longlong2 at = where[k < kTok ? k : 0];
                const long long b = at.x, t = at.y;
                const bool live = on && r < rows && t >= 0;
                const float2* cs = table + (k < kTok ? k : 0) * pairs;
                float x[kVec], y[kVec];
#pragma unroll
                for (int i = 0; i < kVec; ++i) x[i] = y[i] = 0.f;
                if (live) load8<Tx>(static_cast<const Tx*>(s.x) + s.sx.at(b, t, head) + e0, x);
                float inv = 1.f;
                if (p.norm != kNoNorm) {
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < kVec; ++i) ss = fmaf(x[i], x[i], ss);
                    const float m = fmaf(group_sum<G>(ss), n_inv, p.eps);
                    inv = m > 0.f ? 1.f / sqrtf(m) : 0.f;   // a row of zeros without eps stays zero
                }
                if constexpr (!kBackward) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) y[i] = x[i] * (inv * s.scale) * w[i];
                    if (pairs) rotate<G>(y, cs, gl, p.rot, p.layout, p.inverse ? -1.f : 1.f);
                    if (live) store8<Tx>(static_cast<Tx*>(s.out) + s.so.at(b, t, head) + e0, y);
                } else {
                    if (live) load8<Tx>(static_cast<const Tx*>(s.dout) + s.so.at(b, t, head) + e0, y);
                    if (pairs) rotate<G>(y, cs, gl, p.rot, p.layout, -1.f);
                    float dot = 0.f;
#pragma unroll
                    for (int i = 0; i < kVec; ++i) {
                        y[i] *= s.scale;
                        dw[sd][i] = fmaf(y[i], x[i] * inv, dw[sd][i]);
                        y[i] *= w[i];
                        dot = fmaf(y[i], x[i], dot);
                    }
                    dot = p.norm == kNoNorm ? 0.f : group_sum<G>(dot) * (inv * inv * n_inv);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) y[i] = inv * fmaf(-x[i], dot, y[i]);
                    if (live) store8<Tx>(static_cast<Tx*>(s.out) + s.sd.at(b, t, head) + e0, y);
                }
            }
        }
    }
    if constexpr (kBackward) {
#pragma unroll
        for (int sd = 0; sd < 2; ++sd) {
            if (!p.side[sd].dw) continue;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kVec; ++i) sums[group * G * kVec + e0 + i] = dw[sd][i];
            __syncthreads();
            if (threadIdx.x < p.width) {
                float t = 0.f;
                for (int g = 0; g < kGroups; ++g) t += sums[g * G * kVec + threadIdx.x];
                p.side[sd].dw[(size_t)blockIdx.x * p.width + threadIdx.x] = t;
            }
        }
    }
}

// dw of both sides from the CTAs' partial sums, in a fixed order.
__global__ void __launch_bounds__(256) dw_kernel(const float* part_q, const float* part_k, float* dwq, float* dwk,
                                                 int parts, int width) {
    const float* part = blockIdx.y ? part_k : part_q;
    float* dw = blockIdx.y ? dwk : dwq;
    if (!dw) return;
    __shared__ float s[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float t = 0.f;
    if (c < width)
        for (int i = w; i < parts; i += 8) t += part[(size_t)i * width + c];
    s[w][threadIdx.x & 31] = t;
    __syncthreads();
    if (w == 0 && c < width) {
        for (int i = 1; i < 8; ++i) t += s[i][threadIdx.x & 31];
        dw[c] = t;
    }
}

}  // namespace heads
}  // namespace osdn
