// Norms of queries and keys for each head with the position rotation in the same pass, the backward
// of both, and (with the norm off) the rotation alone.
//
// For a row x of one token and head, n = 1 (L2) or its width (RMS):
//   inv = (sum x^2 / n + eps)^(-1/2),  y = scale w inv x,  out = m R(theta) y on the first rot
// features and y on the rest, R turning the pairs (i, i + rot/2) or (2i, 2i+1) by
// theta_i = position * freq_i. Backward, with g = scale (m R(-theta)) dout:
//   dw = sum over rows of g inv x,   dx = inv (g w - x inv^2 / n <g w, x>).
// A row lies in a group of lanes, 8 features a lane, chosen so that both features of a pair are in one lane;
// only a row's sums go between the lanes.
//
// Memory bounds it: 4 bytes an element (bf16) forward for 7 operations. What it takes to get there is few
// instructions a row, 4 rows in flight a lane, and the angles made once a token and shared by its heads.
// Measured, bf16, forward B8 T4096 16 + 16 heads of 128 (L2, rotation) / rotation alone B1 T32768 16 heads:
// a table a CTA and partners by shuffles 188 / 98 us; a warp a token, pairs in one lane 148 / 69; rows by
// stepped pointers and an approximate root 104 / 54; rows loaded ahead of the angles, CTAs that stay
// 100 / 47; a group of lanes a token 94 / 46 us, 88% and 90% of the measured copy rate. What is left is the
// latency of the loads: 4.1 of the 9.5 warps that wait an issue wait for them, at 22 warps an SM (80 registers), and
// issue takes 2.4 of 4 a cycle. Backward at the first size 151 us (82%). fp32, B8 T2048 16 + 16 heads of 128:
// forward 93, with the backward 228 us (89% and 73%).
#pragma once
#include <type_traits>

#include "pairs.cuh"

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
    int parts, part_rows;           // a token's rows in parts of part_rows, a group each
    unsigned blocks;                // CTAs of this side: those of q come first
    float scale;
};

struct Args {
    Side side[2];
    const long long* positions;     // [B, T] or NULL: pos0 + t
    const double* freqs;            // [rot / 2]
    const int* lengths;             // [B] or NULL
    long long pos0;
    unsigned tokens;                // B * T
    int T, width, rot, norm, layout, inverse, zero_rest;
    float eps, amplitude;
};

// A lane's 8 features as four pairs (p_i, q_i) that turn together where the row is rotated: half layout,
// two runs of 4, d apart; interleaved, one run of 8 with its even and odd features apart (d = 4).
struct Eight {
    float2 p[2], q[2];
};
__device__ __forceinline__ float low(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int kLayout, typename T> struct Raw;   // as loaded, not yet converted
template <int kLayout> struct Raw<kLayout, __nv_bfloat16> {
    uint2 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16* at, int d) {
        if (kLayout == kHalf) {
            a = *reinterpret_cast<const uint2*>(at);
            b = *reinterpret_cast<const uint2*>(at + d);
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(at);
            a = make_uint2(u.x, u.y);
            b = make_uint2(u.z, u.w);
        }
    }
    __device__ __forceinline__ void zero() { a = b = make_uint2(0, 0); }
    __device__ __forceinline__ Eight get() const {
        if (kLayout == kHalf)
            return {{make_float2(low(a.x), high(a.x)), make_float2(low(a.y), high(a.y))},
                    {make_float2(low(b.x), high(b.x)), make_float2(low(b.y), high(b.y))}};
        return {{make_float2(low(a.x), low(a.y)), make_float2(low(b.x), low(b.y))},
                {make_float2(high(a.x), high(a.y)), make_float2(high(b.x), high(b.y))}};
    }
};
template <int kLayout> struct Raw<kLayout, float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* at, int d) {
        a = *reinterpret_cast<const float4*>(at);
        b = *reinterpret_cast<const float4*>(at + d);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ Eight get() const {
        if (kLayout == kHalf) return {{make_float2(a.x, a.y), make_float2(a.z, a.w)}, {make_float2(b.x, b.y), make_float2(b.z, b.w)}};
        return {{make_float2(a.x, a.z), make_float2(b.x, b.z)}, {make_float2(a.y, a.w), make_float2(b.y, b.w)}};
    }
};
template <int kLayout> __device__ __forceinline__ void put(__nv_bfloat16* at, int d, const Eight& v) {
    if (kLayout == kHalf) {
        *reinterpret_cast<uint2*>(at) = make_uint2(pack(v.p[0].x, v.p[0].y), pack(v.p[1].x, v.p[1].y));
        *reinterpret_cast<uint2*>(at + d) = make_uint2(pack(v.q[0].x, v.q[0].y), pack(v.q[1].x, v.q[1].y));
    } else {
        *reinterpret_cast<uint4*>(at) = make_uint4(pack(v.p[0].x, v.q[0].x), pack(v.p[0].y, v.q[0].y),
                                                         pack(v.p[1].x, v.q[1].x), pack(v.p[1].y, v.q[1].y));
    }
}
template <int kLayout> __device__ __forceinline__ void put(float* at, int d, const Eight& v) {
    if (kLayout == kHalf) {
        *reinterpret_cast<float4*>(at) = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
        *reinterpret_cast<float4*>(at + d) = make_float4(v.q[0].x, v.q[0].y, v.q[1].x, v.q[1].y);
    } else {
        *reinterpret_cast<float4*>(at) = make_float4(v.p[0].x, v.q[0].x, v.p[0].y, v.q[0].y);
        *reinterpret_cast<float4*>(at + d) = make_float4(v.p[1].x, v.q[1].x, v.p[1].y, v.q[1].y);
    }
}
__device__ __forceinline__ float dot(const Eight& a, const Eight& b) {
    float2 t = mul2(a.p[0], b.p[0]);
    t = fma2(a.p[1], b.p[1], t);
    t = fma2(a.q[0], b.q[0], t);
    t = fma2(a.q[1], b.q[1], t);
    return t.x + t.y;
}

// Sum over the G lanes of a group (every lane of the warp takes part).
template <int G> __device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// m cos and m sin of position * freq: the angle in turns and its whole turns taken off in 64 bits
// (a far position times a frequency leaves no digits of the angle in 32), the rest in 32.
// For bf16 the fast sine and cosine do: within 2^-20 for an angle of up to pi, far below its half step.
template <typename Tx> __device__ __forceinline__ float2 cos_sin(double position, double freq, float amplitude) {
    const double turns = position * freq * 0.15915494309189533577;
    const float part = (float)(turns - rint(turns));
    float s, c;
    if constexpr (sizeof(Tx) == 2) {
        s = __sinf(6.2831853f * part);
        c = __cosf(6.2831853f * part);
    } else {
        sincospif(2.f * part, &s, &c);
    }
    return make_float2(amplitude * c, amplitude * s);
}

// Where a lane's pairs turn: m cos and m sin of the first `turning` of its four pairs.
struct Turn {
    float2 c[2], s[2], ns[2];           // ns = -s
    int turning;
    __device__ __forceinline__ void apply(Eight& v, bool all) const {
        if (all || turning == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 p = fma2(v.q[i], ns[i], mul2(v.p[i], c[i])), q = fma2(v.p[i], s[i], mul2(v.q[i], c[i]));
                v.p[i] = p;
                v.q[i] = q;
            }
        } else if (turning > 0) {       // the end of a rotated part inside the lane (interleaved)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 p = fma2(v.q[i], ns[i], mul2(v.p[i], c[i])), q = fma2(v.p[i], s[i], mul2(v.q[i], c[i]));
                if (2 * i < turning) v.p[i].x = p.x, v.q[i].x = q.x;
                if (2 * i + 1 < turning) v.p[i].y = p.y, v.q[i].y = q.y;
            }
        }
    }
};

// A group of G lanes takes the rows of q, or those of k, of one token, or one of the parts that they come in;
// the groups of a warp take neighbouring tokens. A group makes its token's table of cosines (each angle
// once), each lane keeps its own four for every row, and kRows rows are in flight.
template <int G, int kLayout, bool kBackward, typename Tx>
__global__ void __launch_bounds__(kThreads, kBackward ? 2 : 3) heads_kernel(const Args p) {
    extern __shared__ float2 tables[];              // [groups][rot / 2]
    __shared__ float sums[kBackward ? kThreads * kVec : 1];
    constexpr int kGroups = 32 / G, kRows = 4, kWarps = kThreads / 32;
    const bool of_k = blockIdx.x >= p.side[0].blocks;
    const Side s = of_k ? p.side[1] : p.side[0];
    const unsigned block = of_k ? blockIdx.x - p.side[0].blocks : blockIdx.x;
    const int warp = threadIdx.x >> 5, group = threadIdx.x % 32 / G, gl = threadIdx.x % G;
    const bool on = gl * kVec < p.width, whole = p.width == G * kVec, all_turn = p.rot == p.width;
    const int pairs = p.rot / 2;
    float2* table = tables + threadIdx.x / G * pairs;
    const float n_inv = p.norm == kRms ? 1.f / (float)p.width : 1.f;
    // half layout: the lanes of the rotated part take 4 features of each half, the others 8 in a row
    const bool halves = kLayout == kHalf && gl * kVec < p.rot;
    const int op = halves ? gl * 4 : gl * kVec, d = halves ? pairs : 4;
    Turn turn;
    turn.turning = kLayout == kHalf ? (halves ? 4 : 0) : max(0, min(4, (p.rot - gl * kVec) / 2));
#pragma unroll
    for (int i = 0; i < 2; ++i) turn.c[i] = turn.s[i] = turn.ns[i] = all2(0.f);
    let_next_start();
    wait_for_previous();
    Eight w, dw;
#pragma unroll
    for (int i = 0; i < 2; ++i) w.p[i] = w.q[i] = all2(1.f), dw.p[i] = dw.q[i] = all2(0.f);
    if (on && s.w) {
        Raw<kLayout, float> r;
        r.load(s.w + op, d);
        w = r.get();
    }

    const unsigned items = (p.tokens + kGroups - 1) / kGroups * s.parts;   // below 2^31
    for (unsigned item = block * kWarps + warp; item < items; item += s.blocks * kWarps) {
        const unsigned first = item / s.parts, tok = min(first * kGroups + group, p.tokens - 1);
        const unsigned b = tok / p.T, t = tok - b * p.T;
        const bool there = first * kGroups + group < p.tokens;
        const bool live = there && (!p.lengths || (int)t < p.lengths[b]);
        const bool full_warp = whole && __all_sync(0xffffffffu, live);
        const int h0 = (item - first * s.parts) * s.part_rows, h1 = min(h0 + s.part_rows, s.H);
        const Tok3& to = kBackward ? s.sd : s.so;
        const Tx* xp = static_cast<const Tx*>(s.x) + s.sx.at(b, t, h0) + op;
        const Tx* dp = kBackward ? static_cast<const Tx*>(s.dout) + s.so.at(b, t, h0) + op : nullptr;
        Tx* out = static_cast<Tx*>(s.out) + to.at(b, t, h0) + op;
        // the kRows rows from r0 on; `full`: they are all there, in every group, and every lane has its part of them
        auto rows = [&](int r0, auto full) {
            // rows read, and rows written: those behind a length come out as zeros of zeros
            const int left = on && live ? h1 - r0 : 0, wanted = on && there && (live || p.zero_rest) ? h1 - r0 : 0;
            Raw<kLayout, Tx> xr[kRows];
            [[maybe_unused]] Raw<kLayout, Tx> dr[kBackward ? kRows : 1];
#pragma unroll
            for (int k = 0; k < kRows; ++k, xp += s.sx.h) {
                if (!full) xr[k].zero();
                if (full || k < left) xr[k].load(xp, d);
                if constexpr (kBackward) {
                    if (!full) dr[k].zero();
                    if (full || k < left) dr[k].load(dp, d);
                    dp += s.so.h;
                }
            }
            if (pairs && r0 == h0) {                    // behind the first rows' loads
                const double pos = (double)(p.positions ? p.positions[tok] : p.pos0 + (long long)t);
                __syncwarp();                           // the last token's table has been read
                for (int i = gl; i < pairs; i += G) table[i] = cos_sin<Tx>(pos, p.freqs[i], p.amplitude);
                __syncwarp();
                if (turn.turning) {
                    const float2* mine = table + gl * 4;
                    const int m = turn.turning - 1;
                    const float2 t0 = mine[0], t1 = mine[min(1, m)], t2 = mine[min(2, m)], t3 = mine[min(3, m)];
                    const float sg = kBackward || p.inverse ? -1.f : 1.f;
                    turn.c[0] = make_float2(t0.x, t1.x);
                    turn.c[1] = make_float2(t2.x, t3.x);
                    turn.s[0] = make_float2(sg * t0.y, sg * t1.y);
                    turn.s[1] = make_float2(sg * t2.y, sg * t3.y);
#pragma unroll
                    for (int i = 0; i < 2; ++i) turn.ns[i] = make_float2(-turn.s[i].x, -turn.s[i].y);
                }
            }
#pragma unroll
            for (int k = 0; k < kRows; ++k, out += to.h) {
                if (!full && r0 + k >= h1) break;   // every lane takes part in the sums
                const Eight v = xr[k].get();
                float inv = 1.f;
                if (p.norm != kNoNorm) {
                    const float m = fmaf(group_sum<G>(dot(v, v)), n_inv, p.eps);
                    inv = m < 1.17549435e-38f ? 0.f : rroot(m);   // a row of zeros without eps stays zero, NaN stays NaN
                }
                const float2 inv2 = all2(inv);
                Eight y;
                if constexpr (!kBackward) {
                    const float2 f = all2(inv * s.scale);
#pragma unroll
                    for (int i = 0; i < 2; ++i) y.p[i] = mul2(v.p[i], f), y.q[i] = mul2(v.q[i], f);
                } else {
                    y = dr[k].get();
                    turn.apply(y, all_turn);
                    const float2 f = all2(s.scale);
#pragma unroll
                    for (int i = 0; i < 2; ++i) y.p[i] = mul2(y.p[i], f), y.q[i] = mul2(y.q[i], f);
                    if (s.dw) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            dw.p[i] = fma2(y.p[i], mul2(v.p[i], inv2), dw.p[i]);
                            dw.q[i] = fma2(y.q[i], mul2(v.q[i], inv2), dw.q[i]);
                        }
                    }
                }
                if (s.w) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) y.p[i] = mul2(y.p[i], w.p[i]), y.q[i] = mul2(y.q[i], w.q[i]);
                }
                if constexpr (!kBackward) {
                    turn.apply(y, all_turn);
                } else if (p.norm != kNoNorm) {
                    const float2 g = all2(-group_sum<G>(dot(y, v)) * (inv * inv * n_inv));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        y.p[i] = mul2(inv2, fma2(v.p[i], g, y.p[i]));
                        y.q[i] = mul2(inv2, fma2(v.q[i], g, y.q[i]));
                    }
                }
                if (full || k < wanted) put<kLayout>(out, d, y);
            }
        };
        for (int r0 = h0; r0 < h1; r0 += kRows) {
            if (full_warp && r0 + kRows <= h1) rows(r0, std::true_type{});
            else rows(r0, std::false_type{});
        }
    }
    if constexpr (kBackward) {                      // this CTA's part of dw, groups and warps in order
        if (!s.dw) return;
        if (on) put<kLayout>(sums + (threadIdx.x / G) * G * kVec + op, d, dw);
        __syncthreads();
        if (threadIdx.x < p.width) {
            float t = 0.f;
            for (int g = 0; g < kThreads / G; ++g) t += sums[g * G * kVec + threadIdx.x];
            s.dw[(size_t)block * p.width + threadIdx.x] = t;
        }
    }
}

// dw of both sides from the CTAs' partial sums, in a fixed order: a warp a share of them, then the warps.
__global__ void __launch_bounds__(1024) dw_kernel(const float* part_q, const float* part_k, float* dwq, float* dwk,
                                                  int parts_q, int parts_k, int width) {
    const int parts = blockIdx.y ? parts_k : parts_q;
    const float* part = blockIdx.y ? part_k : part_q;
    float* dw = blockIdx.y ? dwk : dwq;
    __shared__ float s[32][33];
    let_next_start();
    wait_for_previous();
    if (!dw) return;
    const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, w = threadIdx.x >> 5;
    float t = 0.f;
    if (c < width)
#pragma unroll 4
        for (int i = w; i < parts; i += 32) t += part[(size_t)i * width + c];
    s[lane][w] = t;
    __syncthreads();
    t = warp_sum(s[w][lane]);                       // channel w of the block, share by share
    if (lane == 0 && blockIdx.x * 32 + w < width) dw[blockIdx.x * 32 + w] = t;
}

}  // namespace heads
}  // namespace osdn
