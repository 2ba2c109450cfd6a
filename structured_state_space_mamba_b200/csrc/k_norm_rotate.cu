// k_norm_rotate.cu -- RMSNorm of the scan's B and C over dstate and the position
// rotation, one pass each way.
//
// Per token and group, for v = B or C (N values, weight w):
//     n = w v rstd,  rstd = 1 / sqrt(mean v^2 + eps)
//     (o_p, o_q) = (n_p cos - n_q sin, n_p sin + n_q cos) for the rotary / 2 pairs
// and backwards, with dz the cotangent rotated by the opposite angle,
//     dw = sum dz v rstd,  d = dz w,  dv = rstd (d - v rstd^2 mean(d v)).
//
// HBM-bound: a value is read and written once (backwards: two read, one
// written).  A group of lanes takes one token, eight values a lane as two
// vectors of four, laid out so that a lane holds both values of its four
// pairs: nothing but the sums crosses lanes.  The lane forms its four angles
// once and walks the token's groups, B and C side by side, so that sines and
// cosines cost 1 / (2 G) of what they would a row.  Positions may be far: the
// angle is a 64-bit number of turns, and only its fraction becomes fp32.
#include <math.h>

#include "common.cuh"
#include "norm_rotate.h"

namespace ssd {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float *v) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float *p, float *v) {
    const float4 u = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float *v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ void store4(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Sine and cosine of a fraction of a turn in [-1/2, 1/2].  For bf16 storage the
// hardware functions do: their absolute error (2^-20) is far below a bf16 step
// of values of their size.
template <typename T>
__device__ __forceinline__ void sincos_turn(float f, float &s, float &c) {
    if constexpr (sizeof(T) == 2) {
        s = __sinf(6.283185307179586f * f);
        c = __cosf(6.283185307179586f * f);
    } else {
        sincospif(2.f * f, &s, &c);
    }
}

// turns of a position: its fraction, rounded once to fp32
__device__ __forceinline__ float turn_fraction(double pos, double turns) {
    const double t = pos * turns;
    return float(t - rint(t));
}
constexpr double kInvTwoPi = 0.15915494309189533577;

// A lane's eight values: where its two vectors of four lie, and how they pair.
//   half-split: the first at 4q of the pairs' first halves, the second rotary/2
//   further; behind the rotary values, two vectors in a row.
//   interleaved: two vectors in a row; pairs are neighbours.
struct Lane {
    int o0, o1;
    bool active;
};
__device__ __forceinline__ Lane lane_of(const RotateShape &s, int q) {
    Lane l;
    l.active = q * 8 < s.N;
    if (s.interleaved || q * 8 >= s.rotary) {
        l.o0 = q * 8;
        l.o1 = q * 8 + 4;
    } else {
        l.o0 = q * 4;
        l.o1 = s.rotary / 2 + q * 4;
    }
    return l;
}
// pair k of a lane: values a(k) and b(k) of its eight
template <bool INTER>
__device__ __forceinline__ constexpr int pa(int k) { return INTER ? 2 * k : k; }
template <bool INTER>
__device__ __forceinline__ constexpr int pb(int k) { return INTER ? 2 * k + 1 : k + 4; }

// Turns a position by frequency of a lane's four pairs, 4q + k in either order
// (0 behind the rotary values, which turned() leaves alone).
__device__ __forceinline__ void lane_turns(const RotateShape &s, const float *inv_freq, int q, double (&turns)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        turns[k] = 4 * q + k < s.rotary / 2 ? double(__ldg(inv_freq + 4 * q + k)) * kInvTwoPi : 0.0;
}
// The lane's pairs rotated by sign times their angles; `pairs` of the four are.
template <bool INTER>
__device__ __forceinline__ void turn(float (&v)[8], const float (&sn)[4], const float (&cs)[4], int pairs,
                                     float sign) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float a = v[pa<INTER>(k)], b = v[pb<INTER>(k)], s = sign * sn[k];
        if (k < pairs) {
            v[pa<INTER>(k)] = a * cs[k] - b * s;
            v[pb<INTER>(k)] = a * s + b * cs[k];
        }
    }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads)
norm_rotate_kernel(const __grid_constant__ RotateShape s, const T *__restrict__ Bm, const T *__restrict__ Cm,
                   const int64_t *__restrict__ positions, const float *__restrict__ inv_freq,
                   const float *__restrict__ wB, const float *__restrict__ wC, T *__restrict__ Bo,
                   T *__restrict__ Co) {
    const int q = threadIdx.x % s.lanes;
    const Lane l = lane_of(s, q);
    double turns[4];
    lane_turns(s, inv_freq, q, turns);
    const int pairs = s.rotary / 2 - 4 * q;
    float wb[8], wc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int o = e < 4 ? l.o0 + e : l.o1 + e - 4;
        wb[e] = l.active && wB ? __ldg(wB + o) : 1.f;
        wc[e] = l.active && wC ? __ldg(wC + o) : 1.f;
    }
    const float inv_n = 1.f / float(s.N);
    const int per = kThreads / s.lanes;  // tokens of a block at a time
    // whole warps stay in the loop: the sums cross their lanes
    for (int64_t base = int64_t(blockIdx.x) * per; base < s.tokens; base += int64_t(gridDim.x) * per) {
        const int64_t tok = base + threadIdx.x / s.lanes;
        const bool act = l.active && tok < s.tokens;
        const int64_t row = act ? tok / s.T : 0, t = act ? tok - row * s.T : 0;
        const T *xb = Bm + row * s.B_batch + t * s.B_token, *xc = Cm + row * s.C_batch + t * s.C_token;
        const double pos = act ? double(__ldg(positions + tok)) : 0.0;
        float sn[4], cs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sincos_turn<T>(turn_fraction(pos, turns[k]), sn[k], cs[k]);
        for (int g = blockIdx.y; g < s.G; g += gridDim.y) {
            float b[8], c[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = c[e] = 0.f;
            const int64_t gi = int64_t(g) * s.N;
            if (act) {
                load4(xb + gi + l.o0, b);
                load4(xb + gi + l.o1, b + 4);
                load4(xc + gi + l.o0, c);
                load4(xc + gi + l.o1, c + 4);
            }
            float sb = 0.f, sc = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sb = fmaf(b[e], b[e], sb);
                sc = fmaf(c[e], c[e], sc);
            }
            sb = rsqrtf(lanes_sum(sb, s.lanes) * inv_n + s.eps);
            sc = rsqrtf(lanes_sum(sc, s.lanes) * inv_n + s.eps);
            if (!act) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                b[e] *= sb * wb[e];
                c[e] *= sc * wc[e];
            }
            turn<INTER>(b, sn, cs, pairs, 1.f);
            turn<INTER>(c, sn, cs, pairs, 1.f);
            const int64_t o = (tok * s.G + g) * s.N;
            store4(Bo + o + l.o0, b);
            store4(Bo + o + l.o1, b + 4);
            store4(Co + o + l.o0, c);
            store4(Co + o + l.o1, c + 4);
        }
    }
}

// dv of one row from its values x and the cotangent d (rotated back in place);
// adds the row's share to the weight's gradient.
template <bool INTER>
__device__ __forceinline__ void row_backward(const RotateShape &s, float inv_n, const float (&x)[8], float (&d)[8],
                                             const float (&w)[8], const float (&sn)[4], const float (&cs)[4],
                                             int pairs, float (&dw)[8]) {
    turn<INTER>(d, sn, cs, pairs, -1.f);
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        ss = fmaf(x[e], x[e], ss);
        dot = fmaf(d[e] * w[e], x[e], dot);
    }
    const float rstd = rsqrtf(lanes_sum(ss, s.lanes) * inv_n + s.eps);
    const float k = lanes_sum(dot, s.lanes) * inv_n * rstd * rstd;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        dw[e] = fmaf(d[e], x[e] * rstd, dw[e]);
        d[e] = rstd * (d[e] * w[e] - x[e] * k);
    }
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads)
norm_rotate_backward_kernel(const __grid_constant__ RotateShape s, const T *__restrict__ dBo,
                            const T *__restrict__ dCo, const T *__restrict__ Bm, const T *__restrict__ Cm,
                            const int64_t *__restrict__ positions, const float *__restrict__ inv_freq,
                            const float *__restrict__ wB, const float *__restrict__ wC, T *__restrict__ dB,
                            T *__restrict__ dC, float *__restrict__ part) {
    __shared__ float red[kWarps][2][256];
    const int q = threadIdx.x % s.lanes;
    const Lane l = lane_of(s, q);
    double turns[4];
    lane_turns(s, inv_freq, q, turns);
    const int pairs = s.rotary / 2 - 4 * q;
    float wb[8], wc[8], gb[8], gc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int o = e < 4 ? l.o0 + e : l.o1 + e - 4;
        wb[e] = l.active && wB ? __ldg(wB + o) : 1.f;
        wc[e] = l.active && wC ? __ldg(wC + o) : 1.f;
        gb[e] = gc[e] = 0.f;
    }
    const float inv_n = 1.f / float(s.N);
    const int per = kThreads / s.lanes;
    for (int64_t base = int64_t(blockIdx.x) * per; base < s.tokens; base += int64_t(gridDim.x) * per) {
        const int64_t tok = base + threadIdx.x / s.lanes;
        const bool act = l.active && tok < s.tokens;
        const int64_t row = act ? tok / s.T : 0, t = act ? tok - row * s.T : 0;
        const T *xb = Bm + row * s.B_batch + t * s.B_token, *xc = Cm + row * s.C_batch + t * s.C_token;
        const double pos = act ? double(__ldg(positions + tok)) : 0.0;
        float sn[4], cs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sincos_turn<T>(turn_fraction(pos, turns[k]), sn[k], cs[k]);
        for (int g = 0; g < s.G; ++g) {
            float b[8], c[8], db[8], dc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = c[e] = db[e] = dc[e] = 0.f;
            const int64_t gi = int64_t(g) * s.N, o = (tok * s.G + g) * s.N;
            if (act) {
                load4(xb + gi + l.o0, b);
                load4(xb + gi + l.o1, b + 4);
                load4(dBo + o + l.o0, db);
                load4(dBo + o + l.o1, db + 4);
                load4(xc + gi + l.o0, c);
                load4(xc + gi + l.o1, c + 4);
                load4(dCo + o + l.o0, dc);
                load4(dCo + o + l.o1, dc + 4);
            }
            row_backward<INTER>(s, inv_n, b, db, wb, sn, cs, pairs, gb);
            row_backward<INTER>(s, inv_n, c, dc, wc, sn, cs, pairs, gc);
            if (!act) continue;
            store4(dB + o + l.o0, db);
            store4(dB + o + l.o1, db + 4);
            store4(dC + o + l.o0, dc);
            store4(dC + o + l.o1, dc + 4);
        }
    }
    if (!part) return;
    // the block's share of the weights' gradients: lanes of the same values, then warps
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        for (int o = s.lanes; o < 32; o <<= 1) {
            gb[e] += __shfl_xor_sync(0xffffffffu, gb[e], o);
            gc[e] += __shfl_xor_sync(0xffffffffu, gc[e], o);
        }
        if (l.active && (threadIdx.x & 31) < s.lanes) {
            const int o = e < 4 ? l.o0 + e : l.o1 + e - 4;
            red[warp][0][o] = gb[e];
            red[warp][1][o] = gc[e];
        }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < 2 * s.N; o += kThreads) {
        const int which = o >= s.N, j = which ? o - s.N : o;
        float sum = 0.f;
        for (int v = 0; v < kWarps; ++v) sum += red[v][which][j];
        part[int64_t(blockIdx.x) * 2 * s.N + o] = sum;
    }
}

// ---------------------------------------------------------------------------
// any dstate, rotary and alignment: one warp a row of B or C, single values.
// Pair j is on lane j % 32 (at most four a lane), and so are the values behind
// the rotary ones.
// ---------------------------------------------------------------------------
struct Row {
    int64_t tok;
    int g;
    bool isC;
};
__device__ __forceinline__ Row row_of(const RotateShape &s, int64_t r) {
    Row w;
    w.isC = r & 1;
    r >>= 1;
    w.tok = r / s.G;
    w.g = int(r - w.tok * s.G);
    return w;
}
__device__ __forceinline__ void pair_of(const RotateShape &s, int j, int &p, int &q) {
    p = s.interleaved ? 2 * j : j;
    q = s.interleaved ? 2 * j + 1 : j + s.rotary / 2;
}
template <typename T>
__device__ __forceinline__ const T *row_ptr(const RotateShape &s, const T *Bm, const T *Cm, const Row &w) {
    const int64_t b = w.tok / s.T, t = w.tok - b * s.T;
    return (w.isC ? Cm + b * s.C_batch + t * s.C_token : Bm + b * s.B_batch + t * s.B_token) + int64_t(w.g) * s.N;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_rotate_any_kernel(const __grid_constant__ RotateShape s, const T *__restrict__ Bm, const T *__restrict__ Cm,
                       const int64_t *__restrict__ positions, const float *__restrict__ inv_freq,
                       const float *__restrict__ wB, const float *__restrict__ wC, T *__restrict__ Bo,
                       T *__restrict__ Co) {
    const int lane = threadIdx.x & 31;
    const int64_t rows = s.tokens * s.G * 2;
    for (int64_t r = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows; r += int64_t(gridDim.x) * kWarps) {
        const Row w = row_of(s, r);
        const T *x = row_ptr(s, Bm, Cm, w);
        T *o = (w.isC ? Co : Bo) + (w.tok * s.G + w.g) * s.N;
        const float *wt = w.isC ? wC : wB;
        float ss = 0.f;
        for (int n = lane; n < s.N; n += 32) {
            const float v = to_f32<T>(x[n]);
            ss = fmaf(v, v, ss);
        }
        const float rstd = rsqrtf(lanes_sum(ss, 32) / float(s.N) + s.eps);
        const double pos = double(__ldg(positions + w.tok));
        for (int j = lane; j < s.rotary / 2; j += 32) {
            int p, q;
            pair_of(s, j, p, q);
            float sn, cs;
            sincos_turn<T>(turn_fraction(pos, double(__ldg(inv_freq + j)) * kInvTwoPi), sn, cs);
            const float a = to_f32<T>(x[p]) * rstd * (wt ? __ldg(wt + p) : 1.f);
            const float b = to_f32<T>(x[q]) * rstd * (wt ? __ldg(wt + q) : 1.f);
            o[p] = from_f32<T>(a * cs - b * sn);
            o[q] = from_f32<T>(a * sn + b * cs);
        }
        for (int n = s.rotary + lane; n < s.N; n += 32)
            o[n] = from_f32<T>(to_f32<T>(x[n]) * rstd * (wt ? __ldg(wt + n) : 1.f));
    }
}

// A warp's rows all lie on one of B and C (rows step by an even number), so its
// sums for that tensor's weight stay in registers: four pairs and eight values
// behind them a lane.
template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_rotate_backward_any_kernel(const __grid_constant__ RotateShape s, const T *__restrict__ dBo,
                                const T *__restrict__ dCo, const T *__restrict__ Bm, const T *__restrict__ Cm,
                                const int64_t *__restrict__ positions, const float *__restrict__ inv_freq,
                                const float *__restrict__ wB, const float *__restrict__ wC, T *__restrict__ dB,
                                T *__restrict__ dC, float *__restrict__ part) {
    __shared__ float red[kWarps][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int n = lane; n < 256; n += 32) red[warp][n] = 0.f;
    __syncwarp();
    const int64_t rows = s.tokens * s.G * 2;
    for (int64_t r = int64_t(blockIdx.x) * kWarps + warp; r < rows; r += int64_t(gridDim.x) * kWarps) {
        const Row w = row_of(s, r);
        const T *x = row_ptr(s, Bm, Cm, w);
        const int64_t off = (w.tok * s.G + w.g) * s.N;
        const T *d = (w.isC ? dCo : dBo) + off;
        T *o = (w.isC ? dC : dB) + off;
        const float *wt = w.isC ? wC : wB;
        const double pos = double(__ldg(positions + w.tok));
        float ss = 0.f, dot = 0.f;
        float z0[4], z1[4];  // the cotangent, rotated back
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = lane + 32 * k;
            z0[k] = z1[k] = 0.f;
            if (j >= s.rotary / 2) continue;
            int p, q;
            pair_of(s, j, p, q);
            float sn, cs;
            sincos_turn<T>(turn_fraction(pos, double(__ldg(inv_freq + j)) * kInvTwoPi), sn, cs);
            const float d0 = to_f32<T>(d[p]), d1 = to_f32<T>(d[q]), x0 = to_f32<T>(x[p]), x1 = to_f32<T>(x[q]);
            z0[k] = d0 * cs + d1 * sn;
            z1[k] = d1 * cs - d0 * sn;
            ss = fmaf(x0, x0, fmaf(x1, x1, ss));
            dot = fmaf(z0[k] * (wt ? __ldg(wt + p) : 1.f), x0, dot);
            dot = fmaf(z1[k] * (wt ? __ldg(wt + q) : 1.f), x1, dot);
        }
        for (int n = s.rotary + lane; n < s.N; n += 32) {
            const float v = to_f32<T>(x[n]);
            ss = fmaf(v, v, ss);
            dot = fmaf(to_f32<T>(d[n]) * (wt ? __ldg(wt + n) : 1.f), v, dot);
        }
        const float rstd = rsqrtf(lanes_sum(ss, 32) / float(s.N) + s.eps);
        const float m = lanes_sum(dot, 32) / float(s.N) * rstd * rstd;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = lane + 32 * k;
            if (j >= s.rotary / 2) continue;
            int p, q;
            pair_of(s, j, p, q);
            const float x0 = to_f32<T>(x[p]), x1 = to_f32<T>(x[q]);
            red[warp][p] = fmaf(z0[k], x0 * rstd, red[warp][p]);
            red[warp][q] = fmaf(z1[k], x1 * rstd, red[warp][q]);
            o[p] = from_f32<T>(rstd * (z0[k] * (wt ? __ldg(wt + p) : 1.f) - x0 * m));
            o[q] = from_f32<T>(rstd * (z1[k] * (wt ? __ldg(wt + q) : 1.f) - x1 * m));
        }
        for (int n = s.rotary + lane; n < s.N; n += 32) {
            const float v = to_f32<T>(x[n]), z = to_f32<T>(d[n]);
            red[warp][n] = fmaf(z, v * rstd, red[warp][n]);
            o[n] = from_f32<T>(rstd * (z * (wt ? __ldg(wt + n) : 1.f) - v * m));
        }
    }
    if (!part) return;
    __syncthreads();
    // even warps hold B's sums, odd ones C's
    for (int o = threadIdx.x; o < 2 * s.N; o += kThreads) {
        const int which = o >= s.N, j = which ? o - s.N : o;
        float sum = 0.f;
        for (int v = which; v < kWarps; v += 2) sum += red[v][j];
        part[int64_t(blockIdx.x) * 2 * s.N + o] = sum;
    }
}

// the two weights' gradients from the blocks' shares [rows][2][N], in order
__global__ void __launch_bounds__(1024)
weight_sum_kernel(const float *__restrict__ part, int rows, int N, float *__restrict__ dwB,
                  float *__restrict__ dwC) {
    __shared__ float acc[32][33];
    const int o = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (o < 2 * N)
        for (int r = threadIdx.y; r < rows; r += 32) s += __ldg(part + int64_t(r) * 2 * N + o);
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && o < 2 * N) {
        float t = 0.f;
        for (int y = 0; y < 32; ++y) t += acc[y][threadIdx.x];
        float *dst = o < N ? dwB : dwC;
        if (dst) dst[o < N ? o : o - N] = t;
    }
}

// Whether the vector kernels take the shape: rows of whole 8-value lanes, pairs
// that fall on whole vectors, and every row on a vector's alignment.
bool vectors(const RotateShape &s, bool bf16, const void *Bm, const void *Cm) {
    const uintptr_t mask = bf16 ? 7u : 15u;
    return s.N % 8 == 0 && (s.interleaved || s.rotary % 8 == 0) && s.B_batch % 4 == 0 && s.B_token % 4 == 0 &&
           s.C_batch % 4 == 0 && s.C_token % 4 == 0 && (reinterpret_cast<uintptr_t>(Bm) & mask) == 0 &&
           (reinterpret_cast<uintptr_t>(Cm) & mask) == 0;
}

constexpr int64_t kMostBlocks = 148 * 16;  // 16 blocks of 128 threads fill an SM

template <typename T>
cudaError_t forward_typed(const RotateShape &s, const T *Bm, const T *Cm, const int64_t *positions,
                          const float *inv_freq, const float *wB, const float *wC, T *Bo, T *Co, cudaStream_t st) {
    if (vectors(s, sizeof(T) == 2, Bm, Cm)) {
        const int64_t per = kThreads / s.lanes, need = (s.tokens + per - 1) / per;
        const unsigned gx = unsigned(need < kMostBlocks ? need : kMostBlocks);
        // few tokens (a decode step): the groups go to blocks of their own,
        // as long as the GPU has room
        int64_t gy = kMostBlocks / gx;
        if (gy > s.G) gy = s.G;
        const dim3 grid(gx, unsigned(gy < 1 ? 1 : gy));
        if (s.interleaved)
            norm_rotate_kernel<T, true><<<grid, kThreads, 0, st>>>(s, Bm, Cm, positions, inv_freq, wB, wC, Bo, Co);
        else
            norm_rotate_kernel<T, false><<<grid, kThreads, 0, st>>>(s, Bm, Cm, positions, inv_freq, wB, wC, Bo, Co);
    } else {
        const int64_t need = (s.tokens * s.G * 2 + kWarps - 1) / kWarps;
        norm_rotate_any_kernel<T><<<unsigned(need < 4 * kMostBlocks ? need : 4 * kMostBlocks), kThreads, 0, st>>>(
            s, Bm, Cm, positions, inv_freq, wB, wC, Bo, Co);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(const RotateShape &s, int blocks, const T *dBo, const T *dCo, const T *Bm, const T *Cm,
                           const int64_t *positions, const float *inv_freq, const float *wB, const float *wC,
                           T *dB, T *dC, float *part, float *dwB, float *dwC, cudaStream_t st) {
    if (vectors(s, sizeof(T) == 2, Bm, Cm)) {
        if (s.interleaved)
            norm_rotate_backward_kernel<T, true><<<blocks, kThreads, 0, st>>>(s, dBo, dCo, Bm, Cm, positions,
                                                                              inv_freq, wB, wC, dB, dC, part);
        else
            norm_rotate_backward_kernel<T, false><<<blocks, kThreads, 0, st>>>(s, dBo, dCo, Bm, Cm, positions,
                                                                               inv_freq, wB, wC, dB, dC, part);
    } else {
        norm_rotate_backward_any_kernel<T><<<blocks, kThreads, 0, st>>>(s, dBo, dCo, Bm, Cm, positions, inv_freq,
                                                                       wB, wC, dB, dC, part);
    }
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess || !part) return e;
    weight_sum_kernel<<<unsigned((2 * s.N + 31) / 32), dim3(32, 32), 0, st>>>(part, blocks, s.N, dwB, dwC);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rotate(const RotateShape &s, bool bf16, const void *Bm, const void *Cm,
                               const int64_t *positions, const float *inv_freq, const float *wB, const float *wC,
                               void *Bo, void *Co, cudaStream_t st) {
    using H = __nv_bfloat16;
    return bf16 ? forward_typed<H>(s, static_cast<const H *>(Bm), static_cast<const H *>(Cm), positions, inv_freq,
                                   wB, wC, static_cast<H *>(Bo), static_cast<H *>(Co), st)
                : forward_typed<float>(s, static_cast<const float *>(Bm), static_cast<const float *>(Cm), positions,
                                       inv_freq, wB, wC, static_cast<float *>(Bo), static_cast<float *>(Co), st);
}

// Blocks of the backward kernels; each leaves its share of the weights'
// gradients.  Fewer than the forward pass's: a block's share costs 2 N values.
int norm_rotate_backward_blocks(const RotateShape &s) {
    const int64_t per = kThreads / s.lanes, need = (s.tokens + per - 1) / per;
    return int(need < kMostBlocks / 2 ? need : kMostBlocks / 2);
}

cudaError_t launch_norm_rotate_backward(const RotateShape &s, bool bf16, const void *dBo, const void *dCo,
                                        const void *Bm, const void *Cm, const int64_t *positions,
                                        const float *inv_freq, const float *wB, const float *wC, void *dB, void *dC,
                                        float *part, float *dwB, float *dwC, cudaStream_t st) {
    using H = __nv_bfloat16;
    const int blocks = norm_rotate_backward_blocks(s);
    return bf16 ? backward_typed<H>(s, blocks, static_cast<const H *>(dBo), static_cast<const H *>(dCo),
                                    static_cast<const H *>(Bm), static_cast<const H *>(Cm), positions, inv_freq, wB,
                                    wC, static_cast<H *>(dB), static_cast<H *>(dC), part, dwB, dwC, st)
                : backward_typed<float>(s, blocks, static_cast<const float *>(dBo), static_cast<const float *>(dCo),
                                        static_cast<const float *>(Bm), static_cast<const float *>(Cm), positions,
                                        inv_freq, wB, wC, static_cast<float *>(dB), static_cast<float *>(dC), part,
                                        dwB, dwC, st);
}

}  // namespace ssd
