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
// turns are two 64-bit numbers, and only their fraction becomes fp32.
//
// 65536 tokens x 8 groups x 128, bf16, slices of a projection: 96 us on the device,
// 5.6 TB/s.  (With one double an angle it was 93 us, against 125 us with scalar
// arithmetic and a load at a time, 101 us with six blocks an SM, 96 us with eight, whose
// 64 registers spill.)
#include <math.h>

#include "common.cuh"
#include "norm_rotate.h"
#include "tma_host.h"

namespace ssd {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// blocks an SM holds (seven cost the bf16 kernel off the wide vectors 12 spilled bytes
// outside its inner loop, and it is the faster for the loads that they have in flight)
template <typename T> constexpr int kForwardPerSm = sizeof(T) == 2 ? 7 : 5;
constexpr int kBackwardPerSm = 4;
constexpr int kAnyPerSm = 8;

// four values as they lie in memory, and as numbers
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> { using type = uint2; };
template <> struct Raw<float> { using type = float4; };
template <typename T>
__device__ __forceinline__ typename Raw<T>::type fetch4(const T *p) {
    return __ldg(reinterpret_cast<const typename Raw<T>::type *>(p));
}
// The same of two and two values, each pair on its own alignment.
__device__ __forceinline__ uint2 fetch22(const __nv_bfloat16 *p, const __nv_bfloat16 *q) {
    return make_uint2(__ldg(reinterpret_cast<const uint32_t *>(p)), __ldg(reinterpret_cast<const uint32_t *>(q)));
}
__device__ __forceinline__ float4 fetch22(const float *p, const float *q) {
    const float2 a = __ldg(reinterpret_cast<const float2 *>(p)), b = __ldg(reinterpret_cast<const float2 *>(q));
    return make_float4(a.x, a.y, b.x, b.y);
}
// two pairs of neighbours, for the packed fp32 operations
__device__ __forceinline__ void widen4(uint2 u, float2 *v) {
    v[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    v[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void widen4(float4 u, float2 *v) {
    v[0] = make_float2(u.x, u.y);
    v[1] = make_float2(u.z, u.w);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float2 *v) {
    const __nv_bfloat162 a = __float22bfloat162_rn(v[0]), b = __float22bfloat162_rn(v[1]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ void store4(float *p, const float2 *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
}
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(v);
}
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

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

// Turns of a position: the fraction, rounded once to fp32.  A position may have 53 bits
// and as many turns before the point, so both products, freq / (2 pi) and that times the
// position, are formed in two doubles each; what is left out is below 2^-50 of a turn.
// (In one double, an angle was off by 1e-4 at 2^40 and by anything at 2^53.)
constexpr double kInvTwoPi = 0x1.45f306dc9c883p-3, kInvTwoPiLow = -0x1.6b01ec5417056p-57;
__device__ __forceinline__ float turn_fraction(double pos, float freq) {
    asm volatile("" : "+f"(freq));  // both products again for every token, not in registers across them
    const double f = double(freq), hi = f * kInvTwoPi;
    const double lo = __fma_rn(f, kInvTwoPiLow, __fma_rn(f, kInvTwoPi, -hi));
    const double t = pos * hi, rest = __fma_rn(pos, lo, __fma_rn(pos, hi, -t));
    const double turn = (t - rint(t)) + rest;
    return float(turn - rint(turn));
}

// A lane's eight values, v[0 .. 3] in pairs of neighbours: where they lie, and how
// they turn.
//   interleaved: eight in a row; each of v turns in itself.
//   half-split: v[0], v[1] among the pairs' first halves, v[2], v[3] rotary/2 further,
//   so that v[0] turns with v[2] and v[1] with v[3]; behind the rotary values, eight
//   in a row.  WIDE: rotary is a multiple of 8 and the lane's vectors are v[0], v[1]
//   and v[2], v[3].  Otherwise it is one of 4, and a lane may hold two pairs, whose
//   v[1] and v[3] are the first four values behind the rotary ones.
struct Lane {
    int o[4];
    int pairs;  // how many of the lane's four turn (at most 0: none)
    bool active;
};
__device__ __forceinline__ Lane lane_of(const RotateShape &s, int q) {
    Lane l;
    l.active = q * 8 < s.N;
    l.pairs = s.rotary / 2 - 4 * q;
    const bool row = s.interleaved || l.pairs <= 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) l.o[e] = row ? q * 8 + 2 * e : (e < 2 ? 4 * q + 2 * e : s.rotary / 2 + 4 * q + 2 * e - 4);
    if (!s.interleaved && l.pairs == 2) {
        l.o[1] = s.rotary;
        l.o[3] = s.rotary + 2;
    }
    return l;
}
template <bool WIDE, typename T>
__device__ __forceinline__ void fetch_lane(const T *p, const Lane &l, typename Raw<T>::type &u, typename Raw<T>::type &v) {
    if (WIDE) {
        u = fetch4(p + l.o[0]);
        v = fetch4(p + l.o[2]);
    } else {
        u = fetch22(p + l.o[0], p + l.o[1]);
        v = fetch22(p + l.o[2], p + l.o[3]);
    }
}
template <bool WIDE, typename T>
__device__ __forceinline__ void store_lane(T *p, const Lane &l, const float2 (&v)[4]) {
    if (WIDE) {
        store4(p + l.o[0], v);
        store4(p + l.o[2], v + 2);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) store2(p + l.o[e], v[e]);
    }
}

// The frequencies of a lane's four pairs, 4q + k in either order.
__device__ __forceinline__ void lane_freqs(const RotateShape &s, const float *inv_freq, int q, float (&freq)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) freq[k] = 4 * q + k < s.rotary / 2 ? __ldg(inv_freq + 4 * q + k) : 0.f;
}
// Sines and cosines of a lane's pairs at a position: half-split, (0, 1) and (2, 3) as
// they meet the values; interleaved, pair by pair.
template <typename T, bool INTER>
struct Turn {
    float2 cs[INTER ? 4 : 2], sn[INTER ? 4 : 2];
    __device__ __forceinline__ void at(double pos, const float (&freq)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float s, c;
            sincos_turn<T>(turn_fraction(pos, freq[k]), s, c);
            if (INTER) {
                cs[k] = both(c);
                sn[k] = make_float2(-s, s);
            } else {
                (k & 1 ? cs[k / 2].y : cs[k / 2].x) = c;
                (k & 1 ? sn[k / 2].y : sn[k / 2].x) = s;
            }
        }
    }
    // turns the values, or back
    __device__ __forceinline__ void operator()(float2 (&v)[4], int pairs, bool back) const {
        if (INTER) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < pairs) {
                    const float2 s = back ? make_float2(-sn[k].x, -sn[k].y) : sn[k];
                    v[k] = fma(make_float2(v[k].y, v[k].x), s, mul(v[k], cs[k]));
                }
        } else {  // pairs by twos, as rotary / 2 is even
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (2 * k >= pairs) break;
                const float2 a = v[k], b = v[k + 2];
                const float2 s = back ? make_float2(-sn[k].x, -sn[k].y) : sn[k], m = make_float2(-s.x, -s.y);
                v[k] = fma(b, m, mul(a, cs[k]));
                v[k + 2] = fma(a, s, mul(b, cs[k]));
            }
        }
    }
};

// sums of a and b over LANES neighbouring lanes
template <int LANES>
__device__ __forceinline__ void lanes_sum2(float &a, float &b) {
#pragma unroll
    for (int o = LANES >> 1; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
}
__device__ __forceinline__ float square_sum(const float2 (&v)[4]) {
    float2 s = mul(v[0], v[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) s = fma(v[e], v[e], s);
    return s.x + s.y;
}
// a lane's weights, ones without any
__device__ __forceinline__ void lane_weights(const float *w, const Lane &l, float2 (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int o = l.o[e];
        v[e] = l.active && w ? make_float2(__ldg(w + o), __ldg(w + o + 1)) : both(1.f);
    }
}
// where a token's row begins
__device__ __forceinline__ void token_place(const RotateShape &s, int64_t tok, int64_t &ob, int64_t &oc) {
    const int64_t row = s.T == s.tokens ? 0 : tok / s.T, t = tok - row * s.T;
    ob = row * s.B_batch + t * s.B_token;
    oc = row * s.C_batch + t * s.C_token;
}

template <typename T, bool INTER, bool WIDE, int LANES>
__global__ void __launch_bounds__(kThreads, kForwardPerSm<T>)
norm_rotate_kernel(const __grid_constant__ RotateShape s, const T *__restrict__ Bm, const T *__restrict__ Cm,
                   const int64_t *__restrict__ positions, const float *__restrict__ inv_freq,
                   const float *__restrict__ wB, const float *__restrict__ wC, T *__restrict__ Bo,
                   T *__restrict__ Co) {
    constexpr int kPer = kThreads / LANES;  // tokens of a block at a time
    const int q = threadIdx.x % LANES;
    const Lane l = lane_of(s, q);
    float freq[4];
    lane_freqs(s, inv_freq, q, freq);
    float2 wb[4], wc[4];
    lane_weights(wB, l, wb);
    lane_weights(wC, l, wc);
    const float inv_n = 1.f / float(s.N);
    // whole warps stay in the loop: the sums cross their lanes
    for (int64_t base = int64_t(blockIdx.x) * kPer; base < s.tokens; base += int64_t(gridDim.x) * kPer) {
        const int64_t tok = base + threadIdx.x / LANES;
        const bool act = l.active && tok < s.tokens;
        int64_t ob = 0, oc = 0;
        if (act) token_place(s, tok, ob, oc);
        const T *xb = Bm + ob + int64_t(blockIdx.y) * s.N, *xc = Cm + oc + int64_t(blockIdx.y) * s.N;
        const int step = int(gridDim.y) * s.N;
        // the next group's four vectors are on their way while this one's are worked on
        typename Raw<T>::type next[4] = {};
        auto fetch = [&](bool more) {
            if (!act || !more) return;
            fetch_lane<WIDE>(xb, l, next[0], next[1]);
            fetch_lane<WIDE>(xc, l, next[2], next[3]);
            xb += step;
            xc += step;
        };
        fetch(int(blockIdx.y) < s.G);
        Turn<T, INTER> turn;
        turn.at(act ? double(__ldg(positions + tok)) : 0.0, freq);
        int64_t o = (tok * s.G + blockIdx.y) * s.N;
        for (int g = blockIdx.y; g < s.G; g += gridDim.y, o += step) {
            float2 b[4], c[4];
            widen4(next[0], b);
            widen4(next[1], b + 2);
            widen4(next[2], c);
            widen4(next[3], c + 2);
            fetch(g + int(gridDim.y) < s.G);
            float sb = square_sum(b), sc = square_sum(c);
            lanes_sum2<LANES>(sb, sc);
            sb = rsqrtf(fmaf(sb, inv_n, s.eps));
            sc = rsqrtf(fmaf(sc, inv_n, s.eps));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                b[e] = mul(mul(b[e], both(sb)), wb[e]);
                c[e] = mul(mul(c[e], both(sc)), wc[e]);
            }
            turn(b, l.pairs, false);
            turn(c, l.pairs, false);
            if (!act) continue;
            store_lane<WIDE>(Bo + o, l, b);
            store_lane<WIDE>(Co + o, l, c);
        }
    }
}

// dv of one row from its values x, in place of the cotangent d (which is turned
// back first); adds the row's share to the weight's gradient.
template <int LANES, typename TURN>
__device__ __forceinline__ void row_backward(const RotateShape &s, const Lane &l, float inv_n, const TURN &turn,
                                             const float2 (&x)[4], float2 (&d)[4], const float2 (&w)[4],
                                             float2 (&dw)[4]) {
    turn(d, l.pairs, true);
    float2 z[4], t = both(0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        z[e] = mul(d[e], w[e]);
        t = fma(z[e], x[e], t);
    }
    float ss = square_sum(x), dot = t.x + t.y;
    lanes_sum2<LANES>(ss, dot);
    const float rstd = rsqrtf(fmaf(ss, inv_n, s.eps)), k = -dot * inv_n * rstd * rstd;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        dw[e] = fma(d[e], mul(x[e], both(rstd)), dw[e]);
        d[e] = mul(fma(x[e], both(k), z[e]), both(rstd));
    }
}

template <typename T, bool INTER, bool WIDE, int LANES>
__global__ void __launch_bounds__(kThreads, kBackwardPerSm)
norm_rotate_backward_kernel(const __grid_constant__ RotateShape s, const T *__restrict__ dBo,
                            const T *__restrict__ dCo, const T *__restrict__ Bm, const T *__restrict__ Cm,
                            const int64_t *__restrict__ positions, const float *__restrict__ inv_freq,
                            const float *__restrict__ wB, const float *__restrict__ wC, T *__restrict__ dB,
                            T *__restrict__ dC, float *__restrict__ part) {
    constexpr int kPer = kThreads / LANES;
    __shared__ float red[kWarps][2][256];
    const int q = threadIdx.x % LANES;
    const Lane l = lane_of(s, q);
    float freq[4];
    lane_freqs(s, inv_freq, q, freq);
    float2 wb[4], wc[4], gb[4], gc[4];
    lane_weights(wB, l, wb);
    lane_weights(wC, l, wc);
#pragma unroll
    for (int e = 0; e < 4; ++e) gb[e] = gc[e] = both(0.f);
    const float inv_n = 1.f / float(s.N);
    for (int64_t base = int64_t(blockIdx.x) * kPer; base < s.tokens; base += int64_t(gridDim.x) * kPer) {
        const int64_t tok = base + threadIdx.x / LANES;
        const bool act = l.active && tok < s.tokens;
        int64_t ob = 0, oc = 0;
        if (act) token_place(s, tok, ob, oc);
        const T *xb = Bm + ob, *xc = Cm + oc;
        Turn<T, INTER> turn;
        turn.at(act ? double(__ldg(positions + tok)) : 0.0, freq);
        int64_t o = tok * s.G * s.N;
        // while B's row is worked on C's is on its way, and the other way round
        typename Raw<T>::type rb[4] = {}, rc[4] = {};
        auto fetch = [&](const T *x, const T *d, typename Raw<T>::type (&r)[4]) {
            fetch_lane<WIDE>(x, l, r[0], r[1]);
            fetch_lane<WIDE>(d, l, r[2], r[3]);
        };
        auto row = [&](const typename Raw<T>::type (&r)[4], float2 (&x)[4], float2 (&d)[4]) {
            widen4(r[0], x);
            widen4(r[1], x + 2);
            widen4(r[2], d);
            widen4(r[3], d + 2);
        };
        if (act) {
            fetch(xb, dBo + o, rb);
            fetch(xc, dCo + o, rc);
        }
        for (int g = 0; g < s.G; ++g, o += s.N) {
            const bool more = act && g + 1 < s.G;
            float2 x[4], d[4];
            row(rb, x, d);
            xb += s.N;
            if (more) fetch(xb, dBo + o + s.N, rb);
            row_backward<LANES>(s, l, inv_n, turn, x, d, wb, gb);
            if (act) store_lane<WIDE>(dB + o, l, d);
            row(rc, x, d);
            xc += s.N;
            if (more) fetch(xc, dCo + o + s.N, rc);
            row_backward<LANES>(s, l, inv_n, turn, x, d, wc, gc);
            if (act) store_lane<WIDE>(dC + o, l, d);
        }
    }
    if (!part) return;
    // the block's share of the weights' gradients: lanes of the same values, then warps
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float b = e & 1 ? gb[e / 2].y : gb[e / 2].x, c = e & 1 ? gc[e / 2].y : gc[e / 2].x;
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            b += __shfl_xor_sync(0xffffffffu, b, o);
            c += __shfl_xor_sync(0xffffffffu, c, o);
        }
        if (l.active && (threadIdx.x & 31) < LANES) {
            const int o = l.o[e / 2] + (e & 1);
            red[warp][0][o] = b;
            red[warp][1][o] = c;
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
// any dstate, rotary and alignment: one warp a token, row after row of B and C,
// single values.  Pair j is on lane j % 32 (at most four a lane), and so are the
// values behind the rotary ones; the angles are formed once a token.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ void pair_of(const RotateShape &s, int j, int &p, int &q) {
    p = s.interleaved ? 2 * j : j;
    q = s.interleaved ? 2 * j + 1 : j + s.rotary / 2;
}
template <typename T>
__device__ __forceinline__ void any_angles(const RotateShape &s, const float *inv_freq, double pos, int lane,
                                           float (&sn)[4], float (&cs)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (32 * k >= s.rotary / 2) break;
        const int j = lane + 32 * k;
        if (j < s.rotary / 2) sincos_turn<T>(turn_fraction(pos, __ldg(inv_freq + j)), sn[k], cs[k]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_rotate_any_kernel(const __grid_constant__ RotateShape s, const T *__restrict__ Bm, const T *__restrict__ Cm,
                       const int64_t *__restrict__ positions, const float *__restrict__ inv_freq,
                       const float *__restrict__ wB, const float *__restrict__ wC, T *__restrict__ Bo,
                       T *__restrict__ Co) {
    const int lane = threadIdx.x & 31;
    const float inv_n = 1.f / float(s.N);
    for (int64_t tok = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); tok < s.tokens;
         tok += int64_t(gridDim.x) * kWarps) {
        int64_t ob, oc;
        token_place(s, tok, ob, oc);
        float sn[4], cs[4];
        any_angles<T>(s, inv_freq, double(__ldg(positions + tok)), lane, sn, cs);
        for (int row = blockIdx.y; row < 2 * s.G; row += gridDim.y) {  // B's and C's in turn
            const bool isC = row & 1;
            const int64_t at = int64_t(row >> 1) * s.N;
            const T *x = isC ? Cm + oc + at : Bm + ob + at;
            T *o = (isC ? Co : Bo) + tok * s.G * s.N + at;
            const float *wt = isC ? wC : wB;
            float ss = 0.f;
            for (int n = lane; n < s.N; n += 32) {
                const float v = to_f32<T>(x[n]);
                ss = fmaf(v, v, ss);
            }
            const float rstd = rsqrtf(fmaf(warp_sum(ss), inv_n, s.eps));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (32 * k >= s.rotary / 2) break;
                const int j = lane + 32 * k;
                if (j >= s.rotary / 2) continue;
                int p, q;
                pair_of(s, j, p, q);
                const float a = to_f32<T>(x[p]) * rstd * (wt ? __ldg(wt + p) : 1.f);
                const float b = to_f32<T>(x[q]) * rstd * (wt ? __ldg(wt + q) : 1.f);
                o[p] = from_f32<T>(a * cs[k] - b * sn[k]);
                o[q] = from_f32<T>(a * sn[k] + b * cs[k]);
            }
            for (int n = s.rotary + lane; n < s.N; n += 32)
                o[n] = from_f32<T>(to_f32<T>(x[n]) * rstd * (wt ? __ldg(wt + n) : 1.f));
        }
    }
}

// The weights' gradients gather in shared memory, a value always by the same lane.
template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_rotate_backward_any_kernel(const __grid_constant__ RotateShape s, const T *__restrict__ dBo,
                                const T *__restrict__ dCo, const T *__restrict__ Bm, const T *__restrict__ Cm,
                                const int64_t *__restrict__ positions, const float *__restrict__ inv_freq,
                                const float *__restrict__ wB, const float *__restrict__ wC, T *__restrict__ dB,
                                T *__restrict__ dC, float *__restrict__ part) {
    __shared__ float red[kWarps][2][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float inv_n = 1.f / float(s.N);
    for (int n = lane; n < 256; n += 32) red[warp][0][n] = red[warp][1][n] = 0.f;
    __syncwarp();
    for (int64_t tok = int64_t(blockIdx.x) * kWarps + warp; tok < s.tokens; tok += int64_t(gridDim.x) * kWarps) {
        int64_t ob, oc;
        token_place(s, tok, ob, oc);
        float sn[4], cs[4];
        any_angles<T>(s, inv_freq, double(__ldg(positions + tok)), lane, sn, cs);
        for (int row = 0; row < 2 * s.G; ++row) {
            const bool isC = row & 1;
            const int64_t at = int64_t(row >> 1) * s.N, off = tok * s.G * s.N + at;
            const T *x = isC ? Cm + oc + at : Bm + ob + at, *d = (isC ? dCo : dBo) + off;
            T *o = (isC ? dC : dB) + off;
            const float *wt = isC ? wC : wB;
            float *acc = red[warp][isC];
            float ss = 0.f, dot = 0.f;
            float z0[4], z1[4], x0[4], x1[4];  // the cotangent, rotated back, and the values
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (32 * k >= s.rotary / 2) break;
                const int j = lane + 32 * k;
                z0[k] = z1[k] = x0[k] = x1[k] = 0.f;
                if (j >= s.rotary / 2) continue;
                int p, q;
                pair_of(s, j, p, q);
                const float d0 = to_f32<T>(d[p]), d1 = to_f32<T>(d[q]);
                x0[k] = to_f32<T>(x[p]);
                x1[k] = to_f32<T>(x[q]);
                z0[k] = d0 * cs[k] + d1 * sn[k];
                z1[k] = d1 * cs[k] - d0 * sn[k];
                ss = fmaf(x0[k], x0[k], fmaf(x1[k], x1[k], ss));
                dot = fmaf(z0[k] * (wt ? __ldg(wt + p) : 1.f), x0[k], dot);
                dot = fmaf(z1[k] * (wt ? __ldg(wt + q) : 1.f), x1[k], dot);
            }
            for (int n = s.rotary + lane; n < s.N; n += 32) {
                const float v = to_f32<T>(x[n]);
                ss = fmaf(v, v, ss);
                dot = fmaf(to_f32<T>(d[n]) * (wt ? __ldg(wt + n) : 1.f), v, dot);
            }
            const float rstd = rsqrtf(fmaf(warp_sum(ss), inv_n, s.eps));
            const float m = warp_sum(dot) * inv_n * rstd * rstd;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (32 * k >= s.rotary / 2) break;
                const int j = lane + 32 * k;
                if (j >= s.rotary / 2) continue;
                int p, q;
                pair_of(s, j, p, q);
                acc[p] = fmaf(z0[k], x0[k] * rstd, acc[p]);
                acc[q] = fmaf(z1[k], x1[k] * rstd, acc[q]);
                o[p] = from_f32<T>(rstd * (z0[k] * (wt ? __ldg(wt + p) : 1.f) - x0[k] * m));
                o[q] = from_f32<T>(rstd * (z1[k] * (wt ? __ldg(wt + q) : 1.f) - x1[k] * m));
            }
            for (int n = s.rotary + lane; n < s.N; n += 32) {
                const float v = to_f32<T>(x[n]), z = to_f32<T>(d[n]);
                acc[n] = fmaf(z, v * rstd, acc[n]);
                o[n] = from_f32<T>(rstd * (z * (wt ? __ldg(wt + n) : 1.f) - v * m));
            }
        }
    }
    if (!part) return;
    __syncthreads();
    for (int o = threadIdx.x; o < 2 * s.N; o += kThreads) {
        const int which = o >= s.N, j = which ? o - s.N : o;
        float sum = 0.f;
        for (int v = 0; v < kWarps; ++v) sum += red[v][which][j];
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

// How the shape can be read: in vectors of four values, in pairs of them, or one by
// one.  Rows are whole eights either way, pairs of a half-split fall on whole
// vectors (or pairs), and every row lies on their alignment.
enum class Access { kFours, kTwos, kOnes };
Access access_of(const RotateShape &s, bool bf16, const void *Bm, const void *Cm) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(Bm) | reinterpret_cast<uintptr_t>(Cm);
    const int64_t by = s.B_batch | s.B_token | s.C_batch | s.C_token;
    const unsigned es = bf16 ? 2 : 4;
    if (s.N % 8 != 0) return Access::kOnes;
    if ((s.interleaved || s.rotary % 8 == 0) && by % 4 == 0 && at % (4 * es) == 0) return Access::kFours;
    if ((s.interleaved || s.rotary % 4 == 0) && by % 2 == 0 && at % (2 * es) == 0) return Access::kTwos;
    return Access::kOnes;
}

// Calls f with the order of the pairs, the width of an access and the lanes of a
// token as types.
template <typename F>
void by_lanes(const RotateShape &s, Access access, F &&f) {
    auto with = [&](auto inter, auto wide) {
        switch (s.lanes) {
            case 4: return f(inter, wide, std::integral_constant<int, 4>{});
            case 8: return f(inter, wide, std::integral_constant<int, 8>{});
            case 16: return f(inter, wide, std::integral_constant<int, 16>{});
            default: return f(inter, wide, std::integral_constant<int, 32>{});
        }
    };
    auto order = [&](auto wide) { return s.interleaved ? with(std::true_type{}, wide) : with(std::false_type{}, wide); };
    if (access == Access::kFours) order(std::true_type{});
    else order(std::false_type{});
}

// Blocks for `need` portions of work: what the GPU holds at once, every block with
// as many portions as the next (or one fewer).
int64_t even_blocks(int64_t need, int per_sm) {
    const int64_t room = int64_t(device_sm_count()) * per_sm, rounds = (need + room - 1) / room;
    return (need + rounds - 1) / rounds;
}

template <typename T>
cudaError_t forward_typed(const RotateShape &s, const T *Bm, const T *Cm, const int64_t *positions,
                          const float *inv_freq, const float *wB, const float *wC, T *Bo, T *Co, cudaStream_t st) {
    const Access access = access_of(s, sizeof(T) == 2, Bm, Cm);
    if (access != Access::kOnes) {
        const int64_t per = kThreads / s.lanes, need = (s.tokens + per - 1) / per;
        const unsigned gx = unsigned(even_blocks(need, kForwardPerSm<T>));
        // few tokens (a decode step): the groups go to blocks of their own,
        // as long as the GPU has room
        int64_t gy = int64_t(device_sm_count()) * kForwardPerSm<T> / gx;
        if (gy > s.G) gy = s.G;
        const dim3 grid(gx, unsigned(gy < 1 ? 1 : gy));
        by_lanes(s, access, [&](auto inter, auto wide, auto lanes) {
            norm_rotate_kernel<T, decltype(inter)::value, decltype(wide)::value, decltype(lanes)::value>
                <<<grid, kThreads, 0, st>>>(s, Bm, Cm, positions, inv_freq, wB, wC, Bo, Co);
        });
    } else {
        const unsigned gx = unsigned(even_blocks((s.tokens + kWarps - 1) / kWarps, kAnyPerSm));
        int64_t gy = int64_t(device_sm_count()) * kAnyPerSm / gx;
        if (gy > 2 * s.G) gy = 2 * s.G;
        norm_rotate_any_kernel<T><<<dim3(gx, unsigned(gy < 1 ? 1 : gy)), kThreads, 0, st>>>(
            s, Bm, Cm, positions, inv_freq, wB, wC, Bo, Co);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(const RotateShape &s, int blocks, const T *dBo, const T *dCo, const T *Bm, const T *Cm,
                           const int64_t *positions, const float *inv_freq, const float *wB, const float *wC,
                           T *dB, T *dC, float *part, float *dwB, float *dwC, cudaStream_t st) {
    const Access access = access_of(s, sizeof(T) == 2, Bm, Cm);
    if (access != Access::kOnes) {
        by_lanes(s, access, [&](auto inter, auto wide, auto lanes) {
            norm_rotate_backward_kernel<T, decltype(inter)::value, decltype(wide)::value, decltype(lanes)::value>
                <<<blocks, kThreads, 0, st>>>(s, dBo, dCo, Bm, Cm, positions, inv_freq, wB, wC, dB, dC, part);
        });
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

// Blocks of the backward kernels; each leaves its share of the weights' gradients.
int norm_rotate_backward_blocks(const RotateShape &s) {
    const int64_t per = kThreads / s.lanes, need = (s.tokens + per - 1) / per;
    return int(even_blocks(need, kBackwardPerSm));
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
