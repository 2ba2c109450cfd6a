// k_glr.cu -- the gated linear recurrence over whole sequences, its backward
// pass and its decode step.
//
// Per channel, with s(v) = 1 / (1 + e^-v):
//     l_t = A s(r_t),  a_t = e^(l_t),  m_t = sqrt(1 - a_t^2)
//     h_t = a_t h_{t-1} + m_t s(i_t) x_t
// and backwards in time, with K_t = dL/dh_{t-1} through the recurrence alone,
//     G_t = dy_t + K_{t+1},  K_t = a_t G_t.
//
// Either is a scan of pairs (product of decays, sum): a tile of 64 tokens and 64
// channels is read once, its gates are formed in registers, and the tiles of
// one chain (a sequence's chunks for 64 channels) hand the state on through
// global memory in the same launch.  A tile publishes its (product, sum) as
// soon as it has them; a later tile looks back over at most 32 predecessors
// to the nearest one whose outgoing state is known and applies the sums in
// between in their order, so the bits do not depend on how far it looked.
// Tiles are taken by ticket, chunk by chunk over all chains: a tile only ever
// waits for one that a running block holds.
//
// A decay next to one, taken thousands of times, must not be rounded to a
// multiple of 2^-24: everything works with e^l - 1, which keeps its own
// relative precision (the recurrence is h + (e^l - 1) h + u).
#include "common.cuh"
#include "glr.h"
#include "pack8.cuh"
#include "tc_common.cuh"

namespace ssd {

namespace {

// ---------------------------------------------------------------------------
// gates
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rsq(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// the larger of the two, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Gate {
    float sr, si;  // s(r), s(i)
    float cr, ci;  // 1 - s(r), 1 - s(i)
    float l, e1;   // log decay, decay - 1
    float v;       // 1 - decay^2
};

// e^l - 1 for l <= 0: the Taylor sum to l^7 from -1/2 up (the next term is below
// 2^-22 of the result there), the exponential below (where its error is no
// longer magnified by the difference).
__device__ __forceinline__ float decay_minus_1(float l) {
    float p = fmaf(l, 1.f / 5040.f, 1.f / 720.f);
    p = fmaf(l, p, 1.f / 120.f);
    p = fmaf(l, p, 1.f / 24.f);
    p = fmaf(l, p, 1.f / 6.f);
    p = fmaf(l, p, 0.5f);
    p = fmaf(l, p, 1.f);
    p *= l;
    if (l < -0.5f) p = ex2(l * 1.4426950408889634f) - 1.f;
    return p;
}

// One reciprocal serves both sigmoids; the arguments are held at -43 so that
// the product of the two denominators stays finite (s(-43) = 2e-19).
__device__ __forceinline__ Gate gate(float r, float i, float A) {
    Gate g;
    const float er = ex2(max_nan(r, -43.f) * -1.4426950408889634f);
    const float ei = ex2(max_nan(i, -43.f) * -1.4426950408889634f);
    const float q = rcp((1.f + er) * (1.f + ei));
    g.sr = (1.f + ei) * q;
    g.si = (1.f + er) * q;
    g.cr = er * g.sr;
    g.ci = ei * g.si;
    g.l = A * g.sr;
    g.e1 = decay_minus_1(g.l);
    g.v = -g.e1 * (2.f + g.e1);
    return g;
}
// 1 / sqrt(v), 0 for 0
__device__ __forceinline__ float inv_root(float v) { return v == 0.f ? 0.f : rsq(v); }

// ---------------------------------------------------------------------------
// storage: two channels a lane
// ---------------------------------------------------------------------------
// EVEN: the channel count is even, so a lane's pair is one aligned access and
// both channels exist or neither does.
template <typename T, bool EVEN>
__device__ __forceinline__ float2 load2(const T *p, bool a0, bool a1) {
    float2 v = make_float2(0.f, 0.f);
    if (EVEN) {
        if (a0) {
            if constexpr (sizeof(T) == 2) {
                const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(p));
                v = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            } else {
                v = __ldg(reinterpret_cast<const float2 *>(p));
            }
        }
    } else {
        if (a0) v.x = to_f32<T>(p[0]);
        if (a1) v.y = to_f32<T>(p[1]);
    }
    return v;
}
template <typename T, bool EVEN>
__device__ __forceinline__ void store2(T *p, float2 v, bool a0, bool a1) {
    if (EVEN) {
        if (a0) {
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
            else
                *reinterpret_cast<float2 *>(p) = v;
        }
    } else {
        if (a0) p[0] = from_f32<T>(v.x);
        if (a1) p[1] = from_f32<T>(v.y);
    }
}
template <bool EVEN>
__device__ __forceinline__ float2 load_code2(const int8_t *p, float step, bool a0, bool a1) {
    float2 v = make_float2(0.f, 0.f);
    if (EVEN) {
        if (a0) {
            const char2 c = __ldg(reinterpret_cast<const char2 *>(p));
            v = make_float2(float(c.x) * step, float(c.y) * step);
        }
    } else {
        if (a0) v.x = float(p[0]) * step;
        if (a1) v.y = float(p[1]) * step;
    }
    return v;
}
template <bool EVEN>
__device__ __forceinline__ void store_code2(int8_t *p, int c0, int c1, bool a0, bool a1) {
    if (EVEN) {
        if (a0) *reinterpret_cast<char2 *>(p) = make_char2(char(c0), char(c1));
    } else {
        if (a0) p[0] = int8_t(c0);
        if (a1) p[1] = int8_t(c1);
    }
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
struct Tile {
    int tile;      // order of the tile in this launch (its place in the scratch)
    int ct;        // channel tile
    int ntok;      // tokens, 1 .. 64
    int rank;      // tiles of the chain before this one, in the scan's direction
    int stride;    // the previous one of the chain is tile - stride
    int row;       // row of the states
    bool first, last;  // the sequence's first / last chunk
    int64_t tok;   // first token (row * T + offset)
    int64_t chunk; // row of chunk_states
};

// Tickets run over the channel tiles fastest, then over the chains, then along
// them (against time for the backward pass).
__device__ __forceinline__ Tile decode_tile(const GlrShape &s, int tile, bool reverse) {
    Tile t;
    t.tile = tile;
    t.ct = tile % s.nct;
    int g = tile / s.nct;
    int k, nc;
    if (s.nseq == 0) {
        nc = s.nc;
        t.row = g % s.batch;
        k = g / s.batch;
        if (reverse) k = nc - 1 - k;
        t.stride = s.batch * s.nct;
        t.tok = int64_t(t.row) * s.T + int64_t(k) * kGlrChunk;
        t.chunk = int64_t(t.row) * nc + k;
        t.ntok = min(kGlrChunk, s.T - k * kGlrChunk);
    } else {
        if (reverse) g = s.nc - 1 - g;
        int lo = 0, hi = s.nseq;  // the last sequence with cb <= g
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s.cb[mid] <= g) lo = mid; else hi = mid;
        }
        nc = s.cb[lo + 1] - s.cb[lo];
        k = g - s.cb[lo];
        t.row = s.id[lo];
        t.stride = s.nct;
        t.tok = int64_t(s.start[lo]) + k * kGlrChunk;
        t.chunk = s.chunk0 + g;
        t.ntok = min(kGlrChunk, s.len[lo] - k * kGlrChunk);
    }
    t.first = k == 0;
    t.last = k == nc - 1;
    t.rank = reverse ? nc - 1 - k : k;
    return t;
}

__device__ __forceinline__ unsigned int ld_acquire(const unsigned int *f) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(f) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(unsigned int *f, unsigned int v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(f), "r"(v) : "memory");
}

// One warp publishes a tile's sums or its outgoing state.
__device__ __forceinline__ void publish_sums(const GlrScratch &ws, const Tile &t, float2 P, float2 S, int lane) {
    ws.sums[int64_t(t.tile) * 32 + lane] = make_float4(P.x, P.y, S.x, S.y);
    __syncwarp();
    if (lane == 0) st_release(ws.flags + t.tile, 1u);
}
__device__ __forceinline__ void publish_state(const GlrScratch &ws, const Tile &t, float2 h, int lane) {
    ws.state[int64_t(t.tile) * 32 + lane] = h;
    __syncwarp();
    if (lane == 0) st_release(ws.flags + t.tile, 2u);
}

// The state that enters the tile, for one warp (t.rank > 0).  Lane l watches the
// l-th predecessor.  Gives up with the error word set after kWaitLimitNs.
__device__ __forceinline__ bool look_back(const GlrScratch &ws, const Tile &t, int lane, float2 &h,
                                          unsigned int *err) {
    const int window = min(t.rank, 32);
    const unsigned int *f = ws.flags + (t.tile - int64_t(lane + 1) * t.stride);
    int d = 0;
    uint64_t t0 = 0;
    for (uint32_t n = 0;; ++n) {
        const unsigned int v = lane < window ? ld_acquire(f) : 0u;
        const unsigned int done = __ballot_sync(0xffffffffu, v == 2u);
        const unsigned int some = __ballot_sync(0xffffffffu, v != 0u);
        if (done) {
            d = __ffs(done) - 1;
            const unsigned int nearer = (1u << d) - 1u;
            if ((some & nearer) == nearer) break;
        }
        if ((n & 15u) == 15u) {
            const uint64_t now = tc::global_ns();
            if (t0 == 0) t0 = now;
            const bool late = now - t0 > tc::kWaitLimitNs;
            const bool failed = late || (now - t0 > 20000ull && tc::device_failed(err));
            if (__any_sync(0xffffffffu, failed)) {
                if (late && lane == 0 && err) atomicOr(err, 1u);
                return false;
            }
        }
    }
    __syncwarp();
    h = __ldcg(ws.state + (t.tile - int64_t(d + 1) * t.stride) * 32 + lane);
    for (int e = d - 1; e >= 0; --e) {
        const float4 q = __ldcg(ws.sums + (t.tile - int64_t(e + 1) * t.stride) * 32 + lane);
        h.x = fmaf(q.x, h.x, q.z);
        h.y = fmaf(q.y, h.y, q.w);
    }
    return true;
}

// h + e1 h + u
__device__ __forceinline__ float advance(float h, float e1, float u) { return fmaf(e1, h, h) + u; }

constexpr int kWarps = 16;            // warps of a tile
constexpr int kTok = kGlrChunk / kWarps;  // tokens of a warp

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename T>
struct FwdArgs {
    GlrShape s;
    GlrScratch ws;
    const T *x, *r, *i;
    const float *A, *h0;
    T *y;
    float *fin, *states;
    GlrPacked pk;
    unsigned int *err;
};

template <typename T, bool EVEN, bool PACK>
__global__ void __launch_bounds__(kWarps * 32)
glr_forward_kernel(const __grid_constant__ FwdArgs<T> p) {
    __shared__ float4 part[kWarps][32];
    __shared__ float2 hin[32];
    __shared__ int s_tile;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (p.ws.ticket) {
        if (threadIdx.x == 0) s_tile = int(atomicAdd(p.ws.ticket, 1u));
        __syncthreads();
    }
    const Tile t = decode_tile(p.s, p.ws.ticket ? s_tile : int(blockIdx.x), false);
    const int C = p.s.C;
    const int c = t.ct * kGlrCols + 2 * lane;
    const bool a0 = c < C, a1 = c + 1 < C;
    const float A0 = a0 ? __ldg(p.A + c) : 0.f, A1 = a1 ? __ldg(p.A + c + 1) : 0.f;

    float2 xv[kTok], rv[kTok], iv[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
        const int tk = warp * kTok + j;
        const bool ok = tk < t.ntok;
        const int64_t o = (t.tok + tk) * C + c;
        xv[j] = load2<T, EVEN>(p.x + o, ok && a0, ok && a1);
        rv[j] = load2<T, EVEN>(p.r + o, ok && a0, ok && a1);
        iv[j] = load2<T, EVEN>(p.i + o, ok && a0, ok && a1);
    }
    if (PACK) {
        const int64_t cols8 = (C + kPackBlock - 1) / kPackBlock;
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
            const int tk = warp * kTok + j;
            if (tk >= t.ntok) break;
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                const float2 v = n == 0 ? xv[j] : n == 1 ? rv[j] : iv[j];
                const uint32_t m = __reduce_max_sync(0xffffffffu, max(__float_as_uint(v.x) & 0x7fffffffu,
                                                                      __float_as_uint(v.y) & 0x7fffffffu));
                const uint32_t e = pack8_exp(m);
                const float inv = pack8_inv(e);
                store_code2<EVEN>(p.pk.codes[n] + (t.tok + tk) * C + c, pack8_code(v.x, inv),
                                  pack8_code(v.y, inv), a0, a1);
                if (lane == 0) p.pk.exps[n][(t.tok + tk) * cols8 + t.ct] = uint8_t(e);
            }
        }
    }
    float2 e1[kTok], u[kTok];
    float2 P = make_float2(1.f, 1.f), S = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
        const bool ok = warp * kTok + j < t.ntok;
        const Gate g0 = gate(rv[j].x, iv[j].x, A0), g1 = gate(rv[j].y, iv[j].y, A1);
        // behind the sequence's end: the identity
        e1[j].x = ok ? g0.e1 : 0.f;
        e1[j].y = ok ? g1.e1 : 0.f;
        u[j].x = ok ? g0.v * inv_root(g0.v) * g0.si * xv[j].x : 0.f;
        u[j].y = ok ? g1.v * inv_root(g1.v) * g1.si * xv[j].y : 0.f;
        P.x = fmaf(e1[j].x, P.x, P.x);
        P.y = fmaf(e1[j].y, P.y, P.y);
        S.x = advance(S.x, e1[j].x, u[j].x);
        S.y = advance(S.y, e1[j].y, u[j].y);
    }
    part[warp][lane] = make_float4(P.x, P.y, S.x, S.y);
    __syncthreads();
    // the product and sum of the tile's tokens before this warp's
    float2 Pp = make_float2(1.f, 1.f), Sp = make_float2(0.f, 0.f);
    for (int v = 0; v < warp; ++v) {
        const float4 q = part[v][lane];
        Pp.x *= q.x;
        Pp.y *= q.y;
        Sp.x = fmaf(q.x, Sp.x, q.z);
        Sp.y = fmaf(q.y, Sp.y, q.w);
    }
    if (warp == kWarps - 1) {
        const float2 Pt = make_float2(Pp.x * P.x, Pp.y * P.y);
        const float2 St = make_float2(fmaf(P.x, Sp.x, S.x), fmaf(P.y, Sp.y, S.y));
        float2 h = make_float2(0.f, 0.f);
        if (t.first) {
            if (p.h0) h = load2<float, EVEN>(p.h0 + int64_t(t.row) * C + c, a0, a1);
        } else {
            if (!t.last) publish_sums(p.ws, t, Pt, St, lane);
            look_back(p.ws, t, lane, h, p.err);
        }
        const float2 out = make_float2(fmaf(Pt.x, h.x, St.x), fmaf(Pt.y, h.y, St.y));
        if (!t.last) publish_state(p.ws, t, out, lane);
        hin[lane] = h;
        if (p.states) store2<float, EVEN>(p.states + t.chunk * C + c, h, a0, a1);
        if (t.last && p.fin) store2<float, EVEN>(p.fin + int64_t(t.row) * C + c, out, a0, a1);
    }
    __syncthreads();
    float2 h = hin[lane];
    h.x = fmaf(Pp.x, h.x, Sp.x);
    h.y = fmaf(Pp.y, h.y, Sp.y);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
        const int tk = warp * kTok + j;
        if (tk >= t.ntok) break;
        h.x = advance(h.x, e1[j].x, u[j].x);
        h.y = advance(h.y, e1[j].y, u[j].y);
        store2<T, EVEN>(p.y + (t.tok + tk) * C + c, h, a0, a1);
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
template <typename T>
struct BwdArgs {
    GlrShape s;
    GlrScratch ws;
    const T *x, *r, *i, *dy;
    GlrPacked pk;
    const float *A, *states, *dfin;
    T *dx, *dr, *di;
    float *dinit, *dA_part;
    unsigned int *err;
};

template <typename T, bool EVEN, bool PACK>
__global__ void __launch_bounds__(kWarps * 32)
glr_backward_kernel(const __grid_constant__ BwdArgs<T> p) {
    __shared__ float4 part[kWarps][32];   // products, forward sums
    __shared__ float2 rpart[kWarps][32];  // reverse sums, then dA
    __shared__ float2 kin[32];
    __shared__ int s_tile;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (p.ws.ticket) {
        if (threadIdx.x == 0) s_tile = int(atomicAdd(p.ws.ticket, 1u));
        __syncthreads();
    }
    const Tile t = decode_tile(p.s, p.ws.ticket ? s_tile : int(blockIdx.x), true);
    const int C = p.s.C;
    const int c = t.ct * kGlrCols + 2 * lane;
    const bool a0 = c < C, a1 = c + 1 < C;
    const float A0 = a0 ? __ldg(p.A + c) : 0.f, A1 = a1 ? __ldg(p.A + c + 1) : 0.f;
    const float2 h0 = load2<float, EVEN>(p.states + t.chunk * C + c, a0, a1);

    float2 xv[kTok], rv[kTok], iv[kTok], dv[kTok];
    const int64_t cols8 = (C + kPackBlock - 1) / kPackBlock;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
        const int tk = warp * kTok + j;
        const bool ok = tk < t.ntok;
        const int64_t o = (t.tok + tk) * C + c;
        dv[j] = load2<T, EVEN>(p.dy + o, ok && a0, ok && a1);
        if (PACK) {
            const int64_t b = (t.tok + tk) * cols8 + t.ct;
            xv[j] = load_code2<EVEN>(p.pk.codes[0] + o, ok ? pack8_step(__ldg(p.pk.exps[0] + b)) : 0.f, ok && a0, ok && a1);
            rv[j] = load_code2<EVEN>(p.pk.codes[1] + o, ok ? pack8_step(__ldg(p.pk.exps[1] + b)) : 0.f, ok && a0, ok && a1);
            iv[j] = load_code2<EVEN>(p.pk.codes[2] + o, ok ? pack8_step(__ldg(p.pk.exps[2] + b)) : 0.f, ok && a0, ok && a1);
        } else {
            xv[j] = load2<T, EVEN>(p.x + o, ok && a0, ok && a1);
            rv[j] = load2<T, EVEN>(p.r + o, ok && a0, ok && a1);
            iv[j] = load2<T, EVEN>(p.i + o, ok && a0, ok && a1);
        }
    }
    float2 e1[kTok], u[kTok];
    float2 P = make_float2(1.f, 1.f), S = make_float2(0.f, 0.f), R = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
        const bool ok = warp * kTok + j < t.ntok;
        const Gate g0 = gate(rv[j].x, iv[j].x, A0), g1 = gate(rv[j].y, iv[j].y, A1);
        e1[j].x = ok ? g0.e1 : 0.f;
        e1[j].y = ok ? g1.e1 : 0.f;
        u[j].x = ok ? g0.v * inv_root(g0.v) * g0.si * xv[j].x : 0.f;
        u[j].y = ok ? g1.v * inv_root(g1.v) * g1.si * xv[j].y : 0.f;
        P.x = fmaf(e1[j].x, P.x, P.x);
        P.y = fmaf(e1[j].y, P.y, P.y);
        S.x = advance(S.x, e1[j].x, u[j].x);
        S.y = advance(S.y, e1[j].y, u[j].y);
    }
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j) {
        R.x += dv[j].x;
        R.y += dv[j].y;
        R.x = fmaf(e1[j].x, R.x, R.x);
        R.y = fmaf(e1[j].y, R.y, R.y);
    }
    part[warp][lane] = make_float4(P.x, P.y, S.x, S.y);
    rpart[warp][lane] = R;
    __syncthreads();
    // the state before this warp's tokens, and the reverse sums behind them
    float2 h = h0;
    for (int v = 0; v < warp; ++v) {
        const float4 q = part[v][lane];
        h.x = fmaf(q.x, h.x, q.z);
        h.y = fmaf(q.y, h.y, q.w);
    }
    float2 Pp = make_float2(1.f, 1.f), Rp = make_float2(0.f, 0.f);
    for (int v = kWarps - 1; v > warp; --v) {
        const float4 q = part[v][lane];
        const float2 z = rpart[v][lane];
        Pp.x *= q.x;
        Pp.y *= q.y;
        Rp.x = fmaf(q.x, Rp.x, z.x);
        Rp.y = fmaf(q.y, Rp.y, z.y);
    }
    if (warp == 0) {
        const float2 Pt = make_float2(Pp.x * P.x, Pp.y * P.y);
        const float2 Rt = make_float2(fmaf(P.x, Rp.x, R.x), fmaf(P.y, Rp.y, R.y));
        float2 K = make_float2(0.f, 0.f);
        if (t.last) {
            if (p.dfin) K = load2<float, EVEN>(p.dfin + int64_t(t.row) * C + c, a0, a1);
        } else {
            if (!t.first) publish_sums(p.ws, t, Pt, Rt, lane);
            look_back(p.ws, t, lane, K, p.err);
        }
        const float2 out = make_float2(fmaf(Pt.x, K.x, Rt.x), fmaf(Pt.y, K.y, Rt.y));
        if (!t.first) publish_state(p.ws, t, out, lane);
        kin[lane] = K;
        if (t.first && p.dinit) store2<float, EVEN>(p.dinit + int64_t(t.row) * C + c, out, a0, a1);
    }
    __syncthreads();
    float2 K = kin[lane];
    K.x = fmaf(Pp.x, K.x, Rp.x);
    K.y = fmaf(Pp.y, K.y, Rp.y);
    // u[j] becomes the state before the token
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
        const float2 before = h;
        h.x = advance(h.x, e1[j].x, u[j].x);
        h.y = advance(h.y, e1[j].y, u[j].y);
        u[j] = before;
    }
    float2 dA = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j) {
        const int tk = warp * kTok + j;
        const bool ok = tk < t.ntok;
        float dxv[2], drv[2], div[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float A = q ? A1 : A0, xq = q ? xv[j].y : xv[j].x, hq = q ? u[j].y : u[j].x;
            float &Kq = q ? K.y : K.x;
            const Gate g = gate(q ? rv[j].y : rv[j].x, q ? iv[j].y : iv[j].x, A);
            const float rs = inv_root(g.v), m = g.v * rs, a = 1.f + g.e1;
            const float G = (q ? dv[j].y : dv[j].x) + Kq;
            const float six = g.si * xq;
            const float dl = G * a * (hq - a * six * rs);
            dxv[q] = G * m * g.si;
            div[q] = G * m * six * g.ci;
            drv[q] = dl * g.l * g.cr;
            (q ? dA.y : dA.x) += ok ? dl * g.sr : 0.f;
            Kq = ok ? fmaf(g.e1, G, G) : Kq;
        }
        if (!ok) continue;
        const int64_t o = (t.tok + tk) * C + c;
        store2<T, EVEN>(p.dx + o, make_float2(dxv[0], dxv[1]), a0, a1);
        store2<T, EVEN>(p.dr + o, make_float2(drv[0], drv[1]), a0, a1);
        store2<T, EVEN>(p.di + o, make_float2(div[0], div[1]), a0, a1);
    }
    __syncthreads();  // rpart is read above
    rpart[warp][lane] = dA;
    __syncthreads();
    if (warp == 0) {
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            sum.x += rpart[v][lane].x;
            sum.y += rpart[v][lane].y;
        }
        store2<float, EVEN>(p.dA_part + t.chunk * C + c, sum, a0, a1);
    }
}

// Column sums of a [rows, C] array: 32 columns a block, 32 rows at a time, each
// thread in order and then the 32 partial sums in order.
__global__ void __launch_bounds__(1024)
row_sum_kernel(const float *__restrict__ part, int64_t rows, int C, float *__restrict__ out) {
    __shared__ float acc[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < C)
        for (int64_t r = threadIdx.y; r < rows; r += 32) s += __ldg(part + r * C + c);
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < C) {
        float t = 0.f;
        for (int y = 0; y < 32; ++y) t += acc[y][threadIdx.x];
        out[c] = t;
    }
}

// ---------------------------------------------------------------------------
// decode step
// ---------------------------------------------------------------------------
template <typename T, bool EVEN>
__global__ void __launch_bounds__(256)
glr_step_kernel(int batch, int C, const T *__restrict__ x, const T *__restrict__ r, const T *__restrict__ i,
                const float *__restrict__ A, float *__restrict__ state, T *__restrict__ y) {
    const int c = (blockIdx.x * 256 + threadIdx.x) * 2;
    const bool a0 = c < C, a1 = c + 1 < C;
    if (!a0) return;
    const float A0 = __ldg(A + c), A1 = a1 ? __ldg(A + c + 1) : 0.f;
    for (int b = blockIdx.y; b < batch; b += gridDim.y) {
        const int64_t o = int64_t(b) * C + c;
        const float2 xv = load2<T, EVEN>(x + o, a0, a1), rv = load2<T, EVEN>(r + o, a0, a1),
                     iv = load2<T, EVEN>(i + o, a0, a1);
        float2 h;
        if (EVEN) h = *reinterpret_cast<const float2 *>(state + o);
        else h = make_float2(state[o], a1 ? state[o + 1] : 0.f);
        const Gate g0 = gate(rv.x, iv.x, A0), g1 = gate(rv.y, iv.y, A1);
        h.x = advance(h.x, g0.e1, g0.v * inv_root(g0.v) * g0.si * xv.x);
        h.y = advance(h.y, g1.e1, g1.v * inv_root(g1.v) * g1.si * xv.y);
        store2<float, EVEN>(state + o, h, a0, a1);
        store2<T, EVEN>(y + o, h, a0, a1);
    }
}

int64_t tiles_of(const GlrShape &s) { return int64_t(s.nct) * s.nc * (s.nseq ? 1 : s.batch); }

template <typename T, bool EVEN, bool PACK>
cudaError_t forward_typed(const GlrShape &s, const void *x, const void *r, const void *i, const float *A,
                          const float *h0, void *y, float *fin, float *states, const GlrPacked *packed,
                          const GlrScratch &ws, unsigned int *err, cudaStream_t stream) {
    FwdArgs<T> a;
    a.s = s; a.ws = ws;
    a.x = static_cast<const T *>(x); a.r = static_cast<const T *>(r); a.i = static_cast<const T *>(i);
    a.A = A; a.h0 = h0; a.y = static_cast<T *>(y); a.fin = fin; a.states = states;
    a.pk = packed ? *packed : GlrPacked{};
    a.err = err;
    glr_forward_kernel<T, EVEN, PACK><<<unsigned(tiles_of(s)), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, bool EVEN, bool PACK>
cudaError_t backward_typed(const GlrShape &s, const void *x, const void *r, const void *i, const GlrPacked *packed,
                           const float *A, const float *states, const void *dy, const float *dfin, void *dx,
                           void *dr, void *di, float *dinit, float *dA_part, const GlrScratch &ws,
                           unsigned int *err, cudaStream_t stream) {
    BwdArgs<T> a;
    a.s = s; a.ws = ws;
    a.x = static_cast<const T *>(x); a.r = static_cast<const T *>(r); a.i = static_cast<const T *>(i);
    a.dy = static_cast<const T *>(dy);
    a.pk = packed ? *packed : GlrPacked{};
    a.A = A; a.states = states; a.dfin = dfin;
    a.dx = static_cast<T *>(dx); a.dr = static_cast<T *>(dr); a.di = static_cast<T *>(di);
    a.dinit = dinit; a.dA_part = dA_part; a.err = err;
    glr_backward_kernel<T, EVEN, PACK><<<unsigned(tiles_of(s)), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

// Calls f with the storage type and two truth values as types.
template <typename F>
cudaError_t by_type(bool bf16, bool even, bool pack, F &&f) {
    using B = __nv_bfloat16;
    if (bf16)
        return even ? (pack ? f(B{}, std::true_type{}, std::true_type{}) : f(B{}, std::true_type{}, std::false_type{}))
                    : (pack ? f(B{}, std::false_type{}, std::true_type{}) : f(B{}, std::false_type{}, std::false_type{}));
    return even ? (pack ? f(0.f, std::true_type{}, std::true_type{}) : f(0.f, std::true_type{}, std::false_type{}))
                : (pack ? f(0.f, std::false_type{}, std::true_type{}) : f(0.f, std::false_type{}, std::false_type{}));
}

}  // namespace

cudaError_t launch_glr_forward(const GlrShape &s, bool bf16, const void *x, const void *r, const void *i,
                               const float *A, const float *h0, void *y, float *fin, float *states,
                               const GlrPacked *packed, const GlrScratch &ws, unsigned int *err,
                               cudaStream_t stream) {
    return by_type(bf16, s.C % 2 == 0, packed != nullptr, [&](auto t, auto even, auto pack) {
        return forward_typed<decltype(t), decltype(even)::value, decltype(pack)::value>(
            s, x, r, i, A, h0, y, fin, states, packed, ws, err, stream);
    });
}

cudaError_t launch_glr_backward(const GlrShape &s, bool bf16, const void *x, const void *r, const void *i,
                                const GlrPacked *packed, const float *A, const float *states, const void *dy,
                                const float *dfin, void *dx, void *dr, void *di, float *dinit, float *dA_part,
                                const GlrScratch &ws, unsigned int *err, cudaStream_t stream) {
    return by_type(bf16, s.C % 2 == 0, packed != nullptr, [&](auto t, auto even, auto pack) {
        return backward_typed<decltype(t), decltype(even)::value, decltype(pack)::value>(
            s, x, r, i, packed, A, states, dy, dfin, dx, dr, di, dinit, dA_part, ws, err, stream);
    });
}

cudaError_t launch_row_sum(const float *part, int64_t rows, int C, float *out, cudaStream_t stream) {
    row_sum_kernel<<<unsigned((C + 31) / 32), dim3(32, 32), 0, stream>>>(part, rows, C, out);
    return cudaGetLastError();
}

cudaError_t launch_glr_step(int batch, int C, bool bf16, const void *x, const void *r, const void *i,
                            const float *A, float *state, void *y, cudaStream_t stream) {
    const dim3 grid(unsigned((C + 511) / 512), unsigned(batch < 65535 ? batch : 65535));
    return by_type(bf16, C % 2 == 0, false, [&](auto t, auto even, auto) {
        using T = decltype(t);
        glr_step_kernel<T, decltype(even)::value><<<grid, 256, 0, stream>>>(
            batch, C, static_cast<const T *>(x), static_cast<const T *>(r), static_cast<const T *>(i), A, state,
            static_cast<T *>(y));
        return cudaGetLastError();
    });
}

}  // namespace ssd
