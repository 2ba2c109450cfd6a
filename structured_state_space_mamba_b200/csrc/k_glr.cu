// k_glr.cu -- the gated linear recurrence over whole sequences, its backward
// pass and its decode step.
//
// Per channel, with s(v) = 1 / (1 + e^-v):
//     l_t = A s(r_t),  a_t = e^(l_t),  m_t = sqrt(1 - a_t^2)
//     h_t = a_t h_{t-1} + m_t s(i_t) x_t
// and backwards in time, with K_t = dL/dh_{t-1} through the recurrence alone,
//     G_t = dy_t + K_{t+1},  K_t = a_t G_t.
//
// Either is a scan of pairs (decay, sum): a tile of 64 tokens and 64
// channels is read once, its gates are formed in registers, and the tiles of
// one chain (a sequence's chunks for 64 channels) hand the state on through
// global memory in the same launch.  A tile publishes its (decay, sum) as
// soon as it has them; a later tile looks back over at most four predecessors
// to the nearest one whose outgoing state is known and applies the sums in
// between in their order, so the bits do not depend on how far it looked.
// Tiles are taken by ticket, a batch's chunk by chunk over all rows, packed sequences
// one after another: a tile only ever waits for one that a running block holds.
//
// A decay next to one, taken thousands of times, must not be rounded to a
// multiple of 2^-24: the decay of several tokens is the sum of their l until it is
// applied, and applied as e^l - 1.  (As a running product, it was off by 1e-3 after
// 65536 tokens of constant gates, whose roundings all go one way.)  Inside a tile
// a state passes few tokens, and the decay is a factor; 1 - a^2 comes from e^l - 1.
//
// What bounds it.  Compulsory traffic is 8 bytes a value forwards in bf16 and 14
// backwards (11 from checkpoints).  On 4 x 4096 x 5120 the forward pass takes
// 144 us on the device, 4.7 TB/s, the backward pass 309 us (from checkpoints 421 us).
// A pair of channels costs 72 instructions and 8 special functions forwards, 155 and 18
// backwards (212 from checkpoints).  No unit is full: instructions issue in 55 to 58 % of
// the cycles, DRAM is busy for 42 and 36 %.  What passes is latency: most of all
// the wait of a tile for the state before it and, in a block, for the scan warp
// to hand it out.  More warps did not change that (when the forward pass took 140 us:
// four groups of 56 registers 144 us, 16 warps of four tokens 162 us), nor an earlier
// hand-out of the states.  With few chains (1 x 65536 x 2048: 32 of them for 444 groups)
// the tiles of a chain wait for each other's sums through L2: 338 us, 289 us with
// the sums of a tile formed ahead (hold_ahead).
#include "common.cuh"
#include "glr.h"
#include "pack8.cuh"
#include "tc_common.cuh"
#include "tma_host.h"

namespace ssd {

namespace {

// ---------------------------------------------------------------------------
// gates: two channels at a time, in the packed fp32 operations
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
__device__ __forceinline__ float root(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// the larger of the two, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// Operations with a constant are scalar: there it is an immediate, while a packed
// operation needs it in a pair of registers, and moving those there cost a
// quarter of all instructions.  The two constants of the sigmoids are worth
// their registers; an assignment that the compiler cannot see through keeps them.
__device__ __forceinline__ float2 plus(float2 a, float c) { return make_float2(a.x + c, a.y + c); }
__device__ __forceinline__ float2 times_plus(float2 a, float2 b, float c) {
    return make_float2(fmaf(a.x, b.x, c), fmaf(a.y, b.y, c));
}
constexpr float kLog2e = 1.4426950408889634f;
struct Held {
    float2 one, k;  // 1 and -log2(e)
    __device__ __forceinline__ Held() : one(both(1.f)), k(both(-kLog2e)) {
        asm volatile("" : "+f"(one.x), "+f"(one.y), "+f"(k.x), "+f"(k.y));
    }
};

// The argument of a sigmoid: at least -43 (s(-43) = 2e-19), NaN as it is.
__device__ __forceinline__ float2 at_least(float2 v) { return make_float2(max_nan(v.x, -43.f), max_nan(v.y, -43.f)); }
// e^-v, and s(v) from it; 1 - s(v) = e^-v s(v)
__device__ __forceinline__ float2 decayed(const Held &hd, float2 v) {
    const float2 t = mul(v, hd.k);
    return make_float2(ex2(t.x), ex2(t.y));
}
// The two sigmoids of arguments from -43 on by one reciprocal: the product of the
// denominators stays finite.
struct Sig {
    float2 sr, si;  // s(r), s(i)
    float2 er, ei;  // e^-r, e^-i: 1 - s(r) = er * sr
};
__device__ __forceinline__ Sig sigmoids(const Held &hd, float2 r, float2 i) {
    Sig g;
    g.er = decayed(hd, r);
    g.ei = decayed(hd, i);
    const float2 dr = add(g.er, hd.one), di = add(g.ei, hd.one);
    const float2 d = mul(dr, di), q = make_float2(rcp(d.x), rcp(d.y));
    g.sr = mul(di, q);
    g.si = mul(dr, q);
    return g;
}
// e^l - 1 for l from -1/2 to 0: l + l^2 p(l) with p the polynomial of degree 4
// that meets (e^l - 1 - l) / l^2 at the five Chebyshev nodes of [-1/2, 0]: 1.3e-8
// of the result off, at most.
__device__ __forceinline__ float2 decay_minus_1(float2 l) {
    float2 p = make_float2(fmaf(l.x, 0.0011642870f, 0.0082382215f), fmaf(l.y, 0.0011642870f, 0.0082382215f));
    p = times_plus(l, p, 0.0416499302f);
    p = times_plus(l, p, 0.1666656286f);
    p = times_plus(l, p, 0.5f);
    return fma(mul(l, p), l, l);
}
constexpr float kSteep = -0.5f;
// Whether some decay of the warp's channels can be (|l| <= |A|).
__device__ __forceinline__ bool steep_warp(float2 A) { return __any_sync(0xffffffffu, A.x < kSteep || A.y < kSteep); }
// v below there, w from there on
__device__ __forceinline__ float2 by_slope(float2 l, float2 v, float2 w) {
    return make_float2(l.x < kSteep ? v.x : w.x, l.y < kSteep ? v.y : w.y);
}
__device__ __forceinline__ float2 decay_of(float2 l) { return make_float2(ex2(l.x * kLog2e), ex2(l.y * kLog2e)); }
// The decay e^l of a tile as one number q that keeps its own relative precision: e^l - 1
// (at most 0) from l = -1/2 up, e^l itself below, where it is positive: at least 2^-126,
// as what it leaves of a state must not be a difference that is almost the state.
__device__ __forceinline__ float2 decay(float2 l) {
    float2 q = decay_minus_1(l);
    if (__any_sync(0xffffffffu, l.x < kSteep || l.y < kSteep)) {
        const float2 e = decay_of(l);
        q = by_slope(l, make_float2(fmaxf(e.x, 0x1p-126f), fmaxf(e.y, 0x1p-126f)), q);
    }
    return q;
}
// The state behind a tile of that decay which adds S itself.  Rounded to nearest, a state
// that changes by the same fraction of a step at every tile would lose it each time, or
// never move.  So the sum is rounded after a shift of u steps, |u| < 1/2: with the
// multiples of the golden ratio, less whole numbers, for the tiles of a chain
// in turn, as many are rounded up as the fraction asks for, to a few steps
// over any length.  (Costs 4 % on 1 x 65536 x 2048, 280 -> 290 us, and nothing on
// 4 x 4096 x 5120; a second word of the state, handed on with it, took 307 us and 3 %.)
// Where no gate is open nothing is shifted: the state stays as it is.
__device__ __forceinline__ float shift_of(int rank) {
    return (__uint_as_float(0x3f800000u | (uint32_t(rank) * 2654435769u) >> 9) - 1.5f) * 0x1p-23f;  // u 2^-23
}
__device__ __forceinline__ float power_of(float h) { return __uint_as_float(__float_as_uint(h) & 0x7f800000u); }
__device__ __forceinline__ float2 behind(float2 h, float2 q, float2 S, float shift) {
    const float2 u = make_float2(q.x < 0.f ? shift : 0.f, q.y < 0.f ? shift : 0.f);  // no decay, no input
    const float2 base = make_float2(q.x > 0.f ? 0.f : h.x, q.y > 0.f ? 0.f : h.y);
    return add(base, fma(make_float2(power_of(base.x), power_of(base.y)), u, fma(q, h, S)));
}
// The sum of N numbers by pairs: exact where they are all the same.
template <int N>
__device__ __forceinline__ float2 sum_by_pairs(float2 (&v)[N]) {
    static_assert((N & (N - 1)) == 0, "pairs of pairs");
#pragma unroll
    for (int o = 1; o < N; o *= 2)
#pragma unroll
        for (int w = 0; w < N; w += 2 * o) v[w] = add(v[w], v[w + o]);
    return v[0];
}
// a^2 - 1 from a - 1
__device__ __forceinline__ float2 square_minus_1(float2 e1) { return fma(e1, e1, add(e1, e1)); }
// h + e1 h + u
__device__ __forceinline__ float2 advance(float2 h, float2 e1, float2 u) { return add(fma(e1, h, h), u); }
// A token's decay.  Inside a tile the decay a itself does, as a state passes eight of
// them at most (tiles go on from each other by the sum of l), but 1 - a^2 needs
// e^l - 1 where a is next to one.
struct Decay {
    float2 e1;  // e^l - 1
    float2 a;   // precise where e^l - 1 is no longer, below e^-1/2
    float2 w;   // a^2 - 1
};
__device__ __forceinline__ Decay decay_of_token(const Held &hd, float2 l, bool steep) {
    Decay d;
    d.e1 = decay_minus_1(l);
    d.a = add(d.e1, hd.one);
    if (steep) {
        const float2 e = decay_of(l);
        d.e1 = by_slope(l, plus(e, -1.f), d.e1);
        d.a = by_slope(l, e, d.a);
    }
    d.w = square_minus_1(d.e1);
    return d;
}
// Calls f with a truth value as a type.
template <typename F>
__device__ __forceinline__ void by_path(bool v, F &&f) {
    if (v) f(std::true_type{});
    else f(std::false_type{});
}
// l, the decay and what the token brings in, sqrt(1 - a^2) s(i) x, for r and i from -43 on
__device__ __forceinline__ Decay token(const Held &hd, float2 x, float2 r, float2 i, float2 A, bool steep, float2 &l,
                                       float2 &u) {
    const Sig g = sigmoids(hd, r, i);
    l = mul(A, g.sr);
    const Decay d = decay_of_token(hd, l, steep);
    u = mul(make_float2(root(-d.w.x), root(-d.w.y)), mul(g.si, x));
    return d;
}
// 1 / sqrt(-w), 0 for 0 and for what the root takes as 0, numbers below the smallest normal one
__device__ __forceinline__ float inv_root(float w) { return fabsf(w) < 0x1p-126f ? 0.f : rsq(-w); }

// ---------------------------------------------------------------------------
// storage: two channels a lane
// ---------------------------------------------------------------------------
// VEC: rows are whole 16-byte vectors, so a lane's pair is one aligned access and
// both channels exist or neither does.
template <typename T>
__device__ __forceinline__ float2 unpack2(const T *p) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        return *reinterpret_cast<const float2 *>(p);
    }
}
// the same, at least -43: in 16 bits before they are widened
template <typename T>
__device__ __forceinline__ float2 unpack2_at_least(const T *p) {
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 v = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(p), __float2bfloat162_rn(-43.f));
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&v);
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        return at_least(unpack2(p));
    }
}
template <bool VEC>
__device__ __forceinline__ float2 load2(const float *p, bool a0, bool a1) {
    if (VEC) return a0 ? __ldg(reinterpret_cast<const float2 *>(p)) : make_float2(0.f, 0.f);
    return make_float2(a0 ? p[0] : 0.f, a1 ? p[1] : 0.f);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store2(T *p, float2 v, bool a0, bool a1, bool even = false) {
    if (VEC || even) {
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
// A warp's 64 values of one row into the n-th checkpoint, one block of it, two
// values a lane: rows of any length.
__device__ __forceinline__ void pack_row(const GlrPacked &pk, int n, float2 v, int64_t at, int64_t block, int lane,
                                         int c, int C) {
    const uint32_t e = pack8_exp(__reduce_max_sync(
        0xffffffffu, max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu)));
    const float inv = pack8_inv(e);
    if (c < C) pk.codes[n][at] = int8_t(pack8_code(v.x, inv));
    if (c + 1 < C) pk.codes[n][at + 1] = int8_t(pack8_code(v.y, inv));
    if (lane == 0) pk.exps[n][block] = uint8_t(e);
}
// Four rows at once, eight values a lane, eight lanes a block: a third of the
// instructions.  `from`: the lane's eight values in shared memory.
template <typename T>
__device__ __forceinline__ void pack_four(const T *from, int8_t *codes, uint8_t *exps, bool a0, bool a1, bool lead) {
    float v[8];
    uint32_t m;
    if constexpr (sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4 *>(from);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        m = __vmaxu2(__vmaxu2(u[0] & 0x7fff7fffu, u[1] & 0x7fff7fffu),
                     __vmaxu2(u[2] & 0x7fff7fffu, u[3] & 0x7fff7fffu));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = max(m & 0xffff0000u, m << 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(u[e] << 16);
            v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(from), b = *reinterpret_cast<const float4 *>(from + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const uint32_t ex = pack8_exp(m);
    const uint2 q = pack8_eight(v, ex);
    if (sizeof(T) == 2) {  // rows are whole eights
        if (a0) *reinterpret_cast<uint2 *>(codes) = q;
    } else {
        if (a0) reinterpret_cast<uint32_t *>(codes)[0] = q.x;
        if (a1) reinterpret_cast<uint32_t *>(codes)[1] = q.y;
    }
    if (lead && a0) *exps = uint8_t(ex);
}

// ---------------------------------------------------------------------------
// shared memory: a ring of stages, each the raw values of one tile
// ---------------------------------------------------------------------------
template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src, int bytes) {
    const uint32_t d = tc::smem_u32(dst);
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(d), "l"(src), "r"(bytes), "n"(BYTES)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
    bool full;     // 64 tokens of 64 channels
    int64_t tok;   // first token (row * T + offset)
    int64_t base;  // its first value in a [tokens, C] array
    int64_t chunk; // row of chunk_states
};

// n / d by a multiplication (Granlund and Montgomery): n < 2^31, 0 < d < 2^31.
struct Divide {
    uint32_t d, m, s;
    static Divide by(uint32_t d) {
        uint32_t s = 0;
        while ((uint64_t(1) << s) < d) ++s;
        return Divide{d, uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1), s};
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};
struct TileDivide {
    Divide nct, batch;
};

// Tickets run over the channel tiles fastest, then over a batch's rows, then along
// them (against time for the backward pass); packed sequences come one after another,
// each along its chunks.
__device__ __forceinline__ Tile decode_tile(const GlrShape &s, const TileDivide &dv, int tile, bool reverse) {
    Tile t;
    t.tile = tile;
    int g = int(dv.nct(uint32_t(tile)));
    t.ct = tile - g * s.nct;
    int k, nc;
    if (s.nseq == 0) {
        nc = s.nc;
        k = int(dv.batch(uint32_t(g)));
        t.row = g - k * s.batch;
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
    t.full = t.ntok == kGlrChunk && (t.ct + 1) * kGlrCols <= s.C;
    t.base = t.tok * s.C + t.ct * kGlrCols;
    t.rank = reverse ? nc - 1 - k : k;
    return t;
}

// ---------------------------------------------------------------------------
// the hand-off: values that are their own flags
// ---------------------------------------------------------------------------
// The scratch starts as all ones, a NaN that no arithmetic here produces (a
// computed NaN is 0x7fffffff), so a word that differs from it has been written.
// A reader looks at the words it needs themselves: no fence, no flag, one trip
// through L2.
constexpr uint32_t kUnset = 0xffffffffu;

__device__ __forceinline__ void put_sums(const GlrScratch &ws, int tile, int lane, float2 q, float2 S) {
    asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(ws.sums + int64_t(tile) * 32 + lane),
                 "f"(q.x), "f"(q.y), "f"(S.x), "f"(S.y) : "memory");
}
__device__ __forceinline__ void put_state(const GlrScratch &ws, int tile, int lane, float2 h) {
    asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(ws.state + int64_t(tile) * 32 + lane),
                 "f"(h.x), "f"(h.y) : "memory");
}
__device__ __forceinline__ uint32_t get_word(const void *p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float4 get_sums(const GlrScratch &ws, int64_t tile, int lane) {
    float4 v;
    asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(ws.sums + tile * 32 + lane) : "memory");
    return v;
}
__device__ __forceinline__ float2 get_state(const GlrScratch &ws, int64_t tile, int lane) {
    float2 v;
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y)
                 : "l"(ws.state + tile * 32 + lane) : "memory");
    return v;
}
__device__ __forceinline__ bool set(float v) { return __float_as_uint(v) != kUnset; }
__device__ __forceinline__ bool set(float2 v) { return set(v.x) && set(v.y); }
__device__ __forceinline__ bool set(float4 v) { return set(v.x) && set(v.y) && set(v.z) && set(v.w); }

constexpr int kWindow = 4;  // predecessors that a tile looks back over

// The state that enters the tile, for one warp (t.rank > 0): the outgoing state of
// the nearest predecessor that has published it, taken through the sums of those
// in between, in their order.  Every round fetches what is still missing, so that
// a round is one trip through L2, and every lane goes by its own words.  Gives
// up with the error word set after kWaitLimitNs.
template <typename F>
__device__ __forceinline__ bool look_back(const GlrScratch &ws, const Tile &t, int lane, float2 &h,
                                          unsigned int *err, F &&meanwhile) {
    const int window = min(t.rank, kWindow);
    uint64_t t0 = 0;
    float4 sums[kWindow - 1];
    float shift[kWindow - 1];
#pragma unroll
    for (int d = 0; d < kWindow - 1; ++d) {
        sums[d] = make_float4(0.f, 0.f, 0.f, __uint_as_float(kUnset));
        shift[d] = shift_of(t.rank - d - 1);
    }
    for (uint32_t n = 0;; ++n) {
        float2 state[kWindow];
#pragma unroll
        for (int d = 0; d < kWindow; ++d) {
            const int64_t tile = t.tile - int64_t(d + 1) * t.stride;
            state[d] = both(__uint_as_float(kUnset));
            if (d < window) state[d] = get_state(ws, tile, lane);
            if (d < kWindow - 1 && d < window && !set(sums[d])) sums[d] = get_sums(ws, tile, lane);
        }
        bool ok = false;
#pragma unroll
        for (int d = kWindow - 1; d >= 0; --d) ok = set(state[d]) || (d < kWindow - 1 && ok && set(sums[d]));
        if (__all_sync(0xffffffffu, ok)) {
#pragma unroll
            for (int d = kWindow - 1; d >= 0; --d) {
                if (set(state[d])) h = state[d];
                else if (d < kWindow - 1)
                    h = behind(h, make_float2(sums[d].x, sums[d].y), make_float2(sums[d].z, sums[d].w), shift[d]);
            }
            return true;
        }
        meanwhile();
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
}

constexpr int kWarps = 8;                     // compute warps of a tile
constexpr int kGroupThreads = 32 * (kWarps + 1);  // and the scan warp
constexpr int kTok = kGlrChunk / kWarps;      // tokens of a warp
constexpr int kWarpVals = kTok * kGlrCols;

// Copies one warp's tokens of a tile of N [tokens, C] arrays; zeros where there is
// nothing.  The places are the same in all of them and are worked out once.
template <typename T, bool VEC, int N>
__device__ __forceinline__ void fill(T *const (&dst)[N], const T *const (&src)[N], const Tile &t, int C, int warp,
                                     int lane) {
    const int c0 = t.ct * kGlrCols, ntok = t.ntok - warp * kTok;
    if (VEC) {
        constexpr int kBytes = sizeof(T) == 1 ? 8 : 16, kVals = kBytes / sizeof(T), kRow = kGlrCols / kVals;
        constexpr int kRows = 32 / kRow;  // tokens of one step
        const int row = lane / kRow, v = (lane % kRow) * kVals;
        int64_t o = t.base + (int64_t(warp * kTok + row) * C + v);
        if (t.full) {
#pragma unroll
            for (int n = 0; n < kTok / kRows; ++n, o += int64_t(kRows) * C)
#pragma unroll
                for (int a = 0; a < N; ++a)
                    copy_async<kBytes>(dst[a] + n * kRows * kGlrCols + lane * kVals, src[a] + o, kBytes);
            return;
        }
        const bool in = c0 + v < C;
#pragma unroll
        for (int n = 0; n < kTok / kRows; ++n, o += int64_t(kRows) * C) {
            const bool ok = in && row + n * kRows < ntok;
#pragma unroll
            for (int a = 0; a < N; ++a)
                copy_async<kBytes>(dst[a] + n * kRows * kGlrCols + lane * kVals, src[a] + (ok ? o : 0), ok ? kBytes : 0);
        }
    } else if (sizeof(T) == 4) {  // rows of any length still are whole words
#pragma unroll
        for (int n = 0; n < kWarpVals / 32; ++n) {
            const int id = n * 32 + lane, row = id / kGlrCols, v = id % kGlrCols;
            const bool ok = row < ntok && c0 + v < C;
            const int64_t o = ok ? t.base + (int64_t(warp * kTok + row) * C + v) : 0;
#pragma unroll
            for (int a = 0; a < N; ++a) copy_async<4>(dst[a] + id, src[a] + o, ok ? 4 : 0);
        }
    } else if (sizeof(T) == 2 && C % 2 == 0) {  // and so are rows of an even length in 16 bits
        const bool in = c0 + 2 * lane < C;
        int64_t o = t.base + (int64_t(warp * kTok) * C + 2 * lane);
#pragma unroll
        for (int n = 0; n < kTok; ++n, o += C) {
            const bool ok = in && n < ntok;
#pragma unroll
            for (int a = 0; a < N; ++a)
                copy_async<4>(dst[a] + n * kGlrCols + 2 * lane, src[a] + (ok ? o : 0), ok ? 4 : 0);
        }
    } else if (sizeof(T) == 1 && C % 4 == 0) {
        const int row = lane / 16, v = lane % 16 * 4;
        int64_t o = t.base + (int64_t(warp * kTok + row) * C + v);
#pragma unroll
        for (int n = 0; n < kTok; n += 2, o += 2 * int64_t(C)) {
            const bool ok = c0 + v < C && row + n < ntok;
#pragma unroll
            for (int a = 0; a < N; ++a)
                copy_async<4>(dst[a] + (n + row) * kGlrCols + v, src[a] + (ok ? o : 0), ok ? 4 : 0);
        }
    } else {
        // single values, all of a tensor's on their way before the first is stored
#pragma unroll
        for (int a = 0; a < N; ++a) {
            T held[kWarpVals / 32];
#pragma unroll
            for (int n = 0; n < kWarpVals / 32; ++n) {
                const int id = n * 32 + lane, row = id / kGlrCols, v = id % kGlrCols;
                held[n] = row < ntok && c0 + v < C ? src[a][t.base + (int64_t(warp * kTok + row) * C + v)] : T(0.f);
            }
#pragma unroll
            for (int n = 0; n < kWarpVals / 32; ++n) dst[a][n * 32 + lane] = held[n];
        }
    }
}

// Tiles by ticket, or strided over the grid where no state is handed on.
struct Tickets {
    unsigned int *ticket;
    uint32_t tiles, mine, step;  // tiles < 2^31, so that a step past them is a number still
    __device__ __forceinline__ Tickets(unsigned int *t, int n, int groups, int group)
        : ticket(t), tiles(n), mine(group * gridDim.x + blockIdx.x), step(groups * gridDim.x) {}
    // The next tile, raw: what atomicAdd returned, whose first use waits for it.
    __device__ __forceinline__ uint32_t take() {
        if (ticket) return atomicAdd(ticket, 1u);
        const uint32_t n = mine;
        mine = mine > tiles ? mine : mine + step;
        return n - 1u;
    }
    // The ticket word starts at all ones, so a raw ticket is one less than its tile.
    static __device__ __forceinline__ int tile_of(uint32_t raw) { return int(min(raw + 1u, 0x7fffffffu)); }
};

// ---------------------------------------------------------------------------
// a group: compute warps, which never wait for one another, and a scan warp
// ---------------------------------------------------------------------------
// Each compute warp copies, reads and writes its own eight tokens of every tile:
// it forms their gates, leaves their decay and sum, and finishes the tokens
// once it has the state before them.  The scan warp takes the tickets, joins the
// warps' sums, publishes them, looks back and hands every warp its start.  One
// block an SM holds three such groups, which share nothing, so that two of them
// compute while one waits for its state.
//
// Registers decide the shape: 27 warps leave 72 a thread, enough for a tile's
// gates and no more.  Two groups that held two tiles each, to bridge the wait
// themselves, spilled all over their loops; next to this much shared memory L1
// holds few spilled words, and the backward pass took half as long again.  Of the
// kernels as they are, the backward ones from checkpoints and of odd rows in bf16
// spill 28 to 124 bytes, the forward ones of odd rows in bf16 24 to 44.
constexpr int kGroups = 3;
constexpr int kBlock = kGroups * kGroupThreads;

// The tiles of a group, in a ring: a tile's place is set before the starts of an
// earlier one are handed out, with which it becomes visible, and that hand-out is
// waited for before the tile's copies begin.  No ticket is taken earlier than that: a
// group that lags holds up the chains of all the tiles that it has taken.
constexpr int kInfos = 8;
template <int SLOTS>
struct Sync {
    uint64_t parts[SLOTS], ready[SLOTS];
    Tile tile[kInfos];
};
// whether a phase is over, for a whole warp and without waiting
__device__ __forceinline__ bool passed(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred q; mbarrier.test_wait.parity.shared::cta.b64 q, [%1], %2; selp.u32 %0, 1, 0, q; }"
                 : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity) : "memory");
    return __all_sync(0xffffffffu, ok != 0);
}
// The decay of a tile from its warps' sums of l.  (Inside a tile the warps' decays are
// plain numbers: a state passes eight of them at most, and the tile's own state
// goes on from the one before it by this.)
__device__ __forceinline__ float2 join_decay(const float2 (&ls)[kWarps][32], int lane) {
    float2 l[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) l[w] = ls[w][lane];
    return decay(sum_by_pairs(l));
}
// its sum, from the warps' decays and sums
__device__ __forceinline__ float2 join_sum(const float4 (&part)[kWarps][32], int lane) {
    float2 S = both(0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float4 v = part[w][lane];
        S = fma(make_float2(v.x, v.y), S, make_float2(v.z, v.w));
    }
    return S;
}
__device__ __forceinline__ void arrive_warp(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive_cnt(bar, 1);
}

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
    int tiles;
    TileDivide dv;
};
template <typename T, bool HOLD>
struct FwdPlan {
    static constexpr int kStages = sizeof(T) == 2 && !HOLD ? 2 : 1;
    static constexpr int kSlots = HOLD ? 2 : 1;
    static constexpr int kLead = HOLD ? 3 : kStages + 1;  // tiles that are set before the first
    struct Stage {
        T x[kWarpVals], r[kWarpVals], i[kWarpVals];
    };
    struct alignas(128) Smem {
        Stage stage[kStages][kWarps];
        // decays and sums of the warps' tokens; in their place then the states before them
        float4 part[kSlots][kWarps][32];
        float2 l[kSlots][kWarps][32];  // the decays' logarithms
        float4 held[HOLD ? kWarps : 1][HOLD ? kTok : 1][32];
        Sync<kSlots> sync;
        static_assert(kLead + 2 <= kInfos, "a tile's place is taken while it is in use");
    };
    static constexpr int smem = kGroups * sizeof(Smem);
    static_assert(smem <= 227 * 1024, "more shared memory than an SM has");
};

// HOLD: the gates of tile k + 1 are formed, and its sums published, while tile k
// waits for its state; the terms of tile k stay in shared memory meanwhile, in
// place of the second stage of copies (inputs in fp32 leave no room for them).
template <typename T, bool VEC, bool PACK, bool HOLD>
__global__ void __launch_bounds__(kBlock, 1)
glr_forward_kernel(const __grid_constant__ FwdArgs<T> p) {
    using Plan = FwdPlan<T, HOLD>;
    constexpr int NS = Plan::kStages, SL = Plan::kSlots, LEAD = Plan::kLead;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const int group = threadIdx.x / kGroupThreads, lane = threadIdx.x & 31;
    const int warp = (threadIdx.x - group * kGroupThreads) >> 5;
    typename Plan::Smem &sm = reinterpret_cast<typename Plan::Smem *>(smem_raw)[group];
    auto &sync = sm.sync;
    const int C = p.s.C;
    Tickets tickets(p.ws.ticket, p.tiles, kGroups, group);
    auto set_tile = [&](int k, uint32_t raw) {
        const int n = Tickets::tile_of(raw);
        Tile &t = sync.tile[k & (kInfos - 1)];
        if (n < p.tiles) t = decode_tile(p.s, p.dv, n, false);
        else t.tile = -1;
    };
    if (warp == kWarps && lane == 0) {
        for (int n = 0; n < SL; ++n) {
            tc::mbar_init(&sync.parts[n], kWarps);
            tc::mbar_init(&sync.ready[n], 1);
        }
        tc::fence_mbar_init();
        for (int k = 0; k < LEAD; ++k) set_tile(k, tickets.take());
    }
    __syncthreads();

    if (warp == kWarps) {  // the scan warp
        uint32_t next = 0;  // a ticket taken a tile ago
        bool published = false;  // this tile's decay and sum, during the wait of the one before
        float2 q1 = both(0.f), S1 = both(0.f);
        if (lane == 0) next = tickets.take();
        for (int k = 0;; ++k) {
            const Tile &t = sync.tile[k & (kInfos - 1)];
            if (t.tile < 0) break;
            if (lane == 0) set_tile(k + LEAD, next);
            __syncwarp();
            const int c = t.ct * kGlrCols + 2 * lane;
            const bool a0 = c < C, a1 = c + 1 < C;
            float2 h = both(0.f);
            if (!t.first) h = get_state(p.ws, t.tile - int64_t(t.stride), lane);  // it may be there by now
            else if (p.h0) h = load2<VEC>(p.h0 + int64_t(t.row) * C + c, a0, a1);
            auto &part = sm.part[k % SL];
            tc::mbar_wait(&sync.parts[k % SL], (k / SL) & 1, p.err);
            float2 q = q1, S = S1;
            if (!published) {
                q = join_decay(sm.l[k % SL], lane);
                S = join_sum(part, lane);
            }
            if (!t.first && !__all_sync(0xffffffffu, set(h))) {
                if (!t.last && !published) put_sums(p.ws, t.tile, lane, q, S);
                published = false;
                look_back(p.ws, t, lane, h, p.err, [&] {
                    if (SL == 1 || published) return;
                    const Tile &n = sync.tile[(k + 1) & (kInfos - 1)];
                    if (n.tile < 0 || n.first || n.last ||
                        !passed(&sync.parts[(k + 1) % SL], ((k + 1) / SL) & 1))
                        return;
                    q1 = join_decay(sm.l[(k + 1) % SL], lane);
                    S1 = join_sum(sm.part[(k + 1) % SL], lane);
                    put_sums(p.ws, n.tile, lane, q1, S1);
                    published = true;
                });
            } else {
                published = false;
            }
            const float2 out = behind(h, q, S, shift_of(t.rank));
            if (!t.last) put_state(p.ws, t.tile, lane, out);
            const float2 start = h;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 v = part[w][lane];
                *reinterpret_cast<float2 *>(&part[w][lane]) = h;
                h = fma(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
            }
            arrive_warp(&sync.ready[k % SL], lane);
            if (p.states) store2<float, VEC>(p.states + t.chunk * C + c, start, a0, a1);
            if (t.last && p.fin) store2<float, VEC>(p.fin + int64_t(t.row) * C + c, out, a0, a1);
            if (lane == 0) next = tickets.take();
            __syncwarp();
        }
        return;
    }

    auto load = [&](int k) {
        const Tile &t = sync.tile[k & (kInfos - 1)];
        if (t.tile >= 0) {
            typename Plan::Stage &st = sm.stage[k % NS][warp];
            T *const dst[3] = {st.x, st.r, st.i};
            const T *const src[3] = {p.x, p.r, p.i};
            fill<T, VEC, 3>(dst, src, t, C, warp, lane);
        }
        copy_commit();
    };
    auto rates = [&](int k) -> float2 {  // A of tile k
        const Tile &t = sync.tile[k & (kInfos - 1)];
        const int c = t.ct * kGlrCols + 2 * lane;
        return t.tile < 0 ? both(0.f) : load2<VEC>(p.A + c, c < C, c + 1 < C);
    };
    const Held hd;
    // the gates of a tile, and their decay and sum
    auto gates = [&](int k, const Tile &t, float2 A, float2 (&a)[kTok], float2 (&u)[kTok], float4 (&part)[kWarps][32],
                     float2 (&ls)[kWarps][32]) {
        const int ntok = t.ntok - warp * kTok;  // of this warp's tokens
        copy_wait<NS - 1>();
        __syncwarp();
        const typename Plan::Stage &st = sm.stage[k % NS][warp];
        if (PACK) {
            const int64_t cols8 = (C + kPackBlock - 1) / kPackBlock;
            if constexpr (VEC) {
#pragma unroll
                for (int h = 0; h < kTok / 4; ++h) {
                    const int j = 4 * h + lane / 8, v = lane % 8 * 8, c = t.ct * kGlrCols + v;
                    const bool a0 = j < ntok && c < C, a1 = j < ntok && c + 4 < C;
                    const int64_t o = t.base + (int64_t(warp * kTok + j) * C + v);
                    const int64_t block = (t.tok + warp * kTok + j) * cols8 + t.ct;
                    pack_four(st.x + j * kGlrCols + v, p.pk.codes[0] + o, p.pk.exps[0] + block, a0, a1, v == 0);
                    pack_four(st.r + j * kGlrCols + v, p.pk.codes[1] + o, p.pk.exps[1] + block, a0, a1, v == 0);
                    pack_four(st.i + j * kGlrCols + v, p.pk.codes[2] + o, p.pk.exps[2] + block, a0, a1, v == 0);
                }
            } else {
                const int c = t.ct * kGlrCols + 2 * lane;
                int64_t block = (t.tok + warp * kTok) * cols8 + t.ct;
                int64_t o = t.base + (int64_t(warp * kTok) * C + 2 * lane);
#pragma unroll
                for (int j = 0; j < kTok; ++j, block += cols8, o += C) {
                    if (j >= ntok) break;
                    const int at = j * kGlrCols + 2 * lane;
                    pack_row(p.pk, 0, unpack2(st.x + at), o, block, lane, c, C);
                    pack_row(p.pk, 1, unpack2(st.r + at), o, block, lane, c, C);
                    pack_row(p.pk, 2, unpack2(st.i + at), o, block, lane, c, C);
                }
            }
        }
        float2 l[kTok], S = both(0.f);
        by_path(steep_warp(A), [&](auto steep) {
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                const int o = j * kGlrCols + 2 * lane;
                a[j] = token(hd, unpack2(st.x + o), unpack2_at_least(st.r + o), unpack2_at_least(st.i + o), A,
                             decltype(steep)::value, l[j], u[j])
                           .a;
            }
        });
        if (ntok < kTok) {  // behind the sequence's end: the identity
#pragma unroll
            for (int j = 0; j < kTok; ++j)
                if (j >= ntok) {
                    l[j] = u[j] = both(0.f);
                    a[j] = hd.one;
                }
        }
#pragma unroll
        for (int j = 0; j < kTok; ++j) S = fma(a[j], S, u[j]);
        const float2 L = sum_by_pairs(l);
        ls[warp][lane] = L;
        part[warp][lane] = make_float4(ex2(L.x * kLog2e), ex2(L.y * kLog2e), S.x, S.y);
    };
    // a tile's tokens from the state before them; term(j): the decay and the input's part
    auto finish = [&](const Tile &t, const float4 (&part)[kWarps][32], auto term) {
        T *y = p.y + (t.base + (int64_t(warp * kTok) * C + 2 * lane));
        const bool even = C % 2 == 0;
        float2 h = *reinterpret_cast<const float2 *>(&part[warp][lane]);
        if (t.full) {
#pragma unroll
            for (int j = 0; j < kTok; ++j, y += C) {
                const float4 v = term(j);
                h = fma(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
                store2<T, VEC>(y, h, true, true, even);
            }
        } else {
            const int c = t.ct * kGlrCols + 2 * lane, ntok = t.ntok - warp * kTok;
#pragma unroll
            for (int j = 0; j < kTok; ++j, y += C) {
                const float4 v = term(j);
                h = fma(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
                if (j < ntok) store2<T, VEC>(y, h, c < C, c + 1 < C, even);
            }
        }
    };
    for (int k = 0; k < NS; ++k) load(k);
    float2 A = rates(0);
    if constexpr (!HOLD) {
        for (int k = 0;; ++k) {
            const Tile &t = sync.tile[k & (kInfos - 1)];
            if (t.tile < 0) break;
            float2 a[kTok], u[kTok];
            gates(k, t, A, a, u, sm.part[0], sm.l[0]);
            arrive_warp(&sync.parts[0], lane);  // and this warp's part of the stage is read
            load(k + NS);
            A = rates(k + 1);
            tc::mbar_wait(&sync.ready[0], k & 1, p.err);
            finish(t, sm.part[0], [&](int j) { return make_float4(a[j].x, a[j].y, u[j].x, u[j].y); });
        }
    } else {
        for (int k = -1;; ++k) {
            const Tile &t = sync.tile[k & (kInfos - 1)], &n = sync.tile[(k + 1) & (kInfos - 1)];
            if (k >= 0 && t.tile < 0) break;
            const bool more = n.tile >= 0;
            float2 a[kTok], u[kTok];
            if (more) {
                gates(k + 1, n, A, a, u, sm.part[(k + 1) % SL], sm.l[(k + 1) % SL]);
                arrive_warp(&sync.parts[(k + 1) % SL], lane);
                load(k + 2);
                A = rates(k + 2);
            }
            if (k >= 0) {
                tc::mbar_wait(&sync.ready[k % SL], (k / SL) & 1, p.err);
                finish(t, sm.part[k % SL], [&](int j) { return sm.held[warp][j][lane]; });
            }
            if (!more) break;
#pragma unroll
            for (int j = 0; j < kTok; ++j) sm.held[warp][j][lane] = make_float4(a[j].x, a[j].y, u[j].x, u[j].y);
        }
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
    int tiles;
    TileDivide dv;
};
template <typename T, bool PACK>
struct BwdPlan {
    static constexpr int kStages = sizeof(T) == 2 ? (PACK ? 3 : 2) : (PACK ? 2 : 1);
    using In = std::conditional_t<PACK, int8_t, T>;
    struct Stage {
        In in[3][kWarpVals];
        T dy[kWarpVals];
        uint32_t exps[PACK ? 3 : 1][PACK ? kTok : 4];  // the words around the exponent bytes, then the steps
    };
    struct alignas(128) Smem {
        Stage stage[kStages][kWarps];
        // l and forward sums; in their place then the state before the warp's
        // tokens and K behind them
        float4 part[kWarps][32];
        float2 rpart[kWarps][32];  // reverse sums
        float2 dA[2][kWarps][32];
        float2 before[2][32];  // K before the tile's tokens
        Sync<1> sync;
        static_assert(kStages + 2 <= kInfos, "a tile's place is taken while it is in use");
    };
    static constexpr int smem = kGroups * sizeof(Smem);
    static_assert(smem <= 227 * 1024, "more shared memory than an SM has");
};

template <typename T, bool VEC, bool PACK>
__global__ void __launch_bounds__(kBlock, 1)
glr_backward_kernel(const __grid_constant__ BwdArgs<T> p) {
    using Plan = BwdPlan<T, PACK>;
    using In = typename Plan::In;
    constexpr int NS = Plan::kStages;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const int group = threadIdx.x / kGroupThreads, lane = threadIdx.x & 31;
    const int warp = (threadIdx.x - group * kGroupThreads) >> 5;
    typename Plan::Smem &sm = reinterpret_cast<typename Plan::Smem *>(smem_raw)[group];
    auto &sync = sm.sync;
    const int C = p.s.C;
    const int64_t cols8 = (C + kPackBlock - 1) / kPackBlock;
    Tickets tickets(p.ws.ticket, p.tiles, kGroups, group);
    auto set_tile = [&](int k, uint32_t raw) {
        const int n = Tickets::tile_of(raw);
        Tile &t = sync.tile[k & (kInfos - 1)];
        if (n < p.tiles) t = decode_tile(p.s, p.dv, n, true);
        else t.tile = -1;
    };
    if (warp == kWarps && lane == 0) {
        tc::mbar_init(&sync.parts[0], kWarps);
        tc::mbar_init(&sync.ready[0], 1);
        tc::fence_mbar_init();
        for (int k = 0; k < NS + 1; ++k) set_tile(k, tickets.take());
    }
    __syncthreads();

    if (warp == kWarps) {  // the scan warp
        // dA and dinit of tile k, which its warps have left by the time they leave the sums of tile k + 1
        auto sum_dA = [&](int k) {
            const Tile &t = sync.tile[k & (kInfos - 1)];
            const int c = t.ct * kGlrCols + 2 * lane;
            float2 sum = sm.dA[k & 1][0][lane];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) sum = add(sum, sm.dA[k & 1][w][lane]);
            store2<float, VEC>(p.dA_part + t.chunk * C + c, sum, c < C, c + 1 < C);
            // (the tile's own sums have decays far below one only as e^l - 1)
            if (t.first && p.dinit)
                store2<float, VEC>(p.dinit + int64_t(t.row) * C + c, sm.before[k & 1][lane], c < C, c + 1 < C);
        };
        uint32_t next = 0;  // a ticket taken a tile ago
        if (lane == 0) next = tickets.take();
        int k = 0;
        for (;; ++k) {
            const Tile &t = sync.tile[k & (kInfos - 1)];
            if (t.tile < 0) break;
            if (lane == 0) set_tile(k + NS + 1, next);
            __syncwarp();
            const int c = t.ct * kGlrCols + 2 * lane;
            const bool a0 = c < C, a1 = c + 1 < C;
            float2 h = load2<VEC>(p.states + t.chunk * C + c, a0, a1), K = both(0.f);
            if (!t.last) K = get_state(p.ws, t.tile - int64_t(t.stride), lane);
            else if (p.dfin) K = load2<VEC>(p.dfin + int64_t(t.row) * C + c, a0, a1);
            tc::mbar_wait(&sync.parts[0], k & 1, p.err);
            float2 l[kWarps], f[kWarps], R = both(0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                l[w] = *reinterpret_cast<const float2 *>(&sm.part[w][lane]);
                f[w] = make_float2(ex2(l[w].x * kLog2e), ex2(l[w].y * kLog2e));
            }
            const float2 q = decay(sum_by_pairs(l));
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) R = fma(f[w], R, sm.rpart[w][lane]);
            if (!t.last && !__all_sync(0xffffffffu, set(K))) {
                if (!t.first) put_sums(p.ws, t.tile, lane, q, R);
                look_back(p.ws, t, lane, K, p.err, [] {});
            }
            if (!t.first) put_state(p.ws, t.tile, lane, behind(K, q, R, shift_of(t.rank)));
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 v = sm.part[w][lane];
                *reinterpret_cast<float2 *>(&sm.part[w][lane]) = h;
                h = fma(f[w], h, make_float2(v.z, v.w));
            }
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                reinterpret_cast<float2 *>(&sm.part[w][lane])[1] = K;
                K = fma(f[w], K, sm.rpart[w][lane]);
            }
            arrive_warp(&sync.ready[0], lane);
            if (k >= 1) sum_dA(k - 1);
            __syncwarp();
            if (lane == 0) next = tickets.take();
            __syncwarp();
        }
        if (k > 0) {  // the last tile: its warps say when they are through
            tc::mbar_wait(&sync.parts[0], k & 1, p.err);
            sum_dA(k - 1);
        }
        return;
    }

    auto load = [&](int k) {
        const Tile &t = sync.tile[k & (kInfos - 1)];
        if (t.tile >= 0) {
            typename Plan::Stage &st = sm.stage[k % NS][warp];
            if constexpr (PACK) {
                int8_t *const dst[3] = {st.in[0], st.in[1], st.in[2]};
                const int8_t *const src[3] = {p.pk.codes[0], p.pk.codes[1], p.pk.codes[2]};
                fill<int8_t, VEC, 3>(dst, src, t, C, warp, lane);
                T *const ddst[1] = {st.dy};
                const T *const dsrc[1] = {p.dy};
                fill<T, VEC, 1>(ddst, dsrc, t, C, warp, lane);
                // the aligned word around each exponent byte, as far as the array goes
                if (lane < 3 * kTok) {
                    const int n = lane / kTok, row = warp * kTok + lane % kTok;
                    const uint8_t *e = n == 0 ? p.pk.exps[0] : n == 1 ? p.pk.exps[1] : p.pk.exps[2];
                    const int64_t all = int64_t(p.s.batch) * p.s.T * cols8;
                    const int64_t at = row < t.ntok ? ((t.tok + row) * cols8 + t.ct) & ~int64_t(3) : 0;
                    copy_async<4>(&st.exps[n][lane % kTok], e + at, int(all - at < 4 ? all - at : 4));
                }
            } else {
                T *const dst[4] = {st.in[0], st.in[1], st.in[2], st.dy};
                const T *const src[4] = {p.x, p.r, p.i, p.dy};
                fill<T, VEC, 4>(dst, src, t, C, warp, lane);
            }
        }
        copy_commit();
    };
    auto rates = [&](int k) -> float2 {  // A of tile k
        const Tile &t = sync.tile[k & (kInfos - 1)];
        const int c = t.ct * kGlrCols + 2 * lane;
        return t.tile < 0 ? both(0.f) : load2<VEC>(p.A + c, c < C, c + 1 < C);
    };
    const Held hd;
    for (int k = 0; k < NS; ++k) load(k);
    float2 A = rates(0);
    int k = 0;
    for (;; ++k) {
        const Tile &t = sync.tile[k & (kInfos - 1)];
        if (t.tile < 0) break;
        const bool steep = steep_warp(A);
        const int ntok = t.ntok - warp * kTok;
        copy_wait<NS - 1>();
        __syncwarp();
        typename Plan::Stage &st = sm.stage[k % NS][warp];
        if constexpr (PACK) {
            if (lane < 3 * kTok) {
                const int n = lane / kTok, j = lane % kTok;
                const uint32_t shift = 8 * (uint32_t((t.tok + warp * kTok + j) * cols8 + t.ct) & 3u);
                st.exps[n][j] = __float_as_uint(pack8_step((st.exps[n][j] >> shift) & 255u));
            }
            __syncwarp();
        }
        // x, r or i of token j of this warp
        auto input = [&](int n, int j) -> float2 {
            const int o = j * kGlrCols + 2 * lane;
            if constexpr (PACK) {
                return unpack8_two(*reinterpret_cast<const uint16_t *>(st.in[n] + o), __uint_as_float(st.exps[n][j]));
            } else {
                return unpack2(st.in[n] + o);
            }
        };
        auto gate = [&](int n, int j) -> float2 {  // r or i, at least -43
            if constexpr (PACK) return at_least(input(n, j));
            else return unpack2_at_least(st.in[n] + j * kGlrCols + 2 * lane);
        };
        auto cotangent = [&](int j) -> float2 { return unpack2(st.dy + j * kGlrCols + 2 * lane); };
        float2 e1[kTok], u[kTok];
        {
            float2 l[kTok], S = both(0.f), R = both(0.f);
#pragma unroll
            for (int j = 0; j < kTok; ++j)
                e1[j] = token(hd, input(0, j), gate(1, j), gate(2, j), A, steep, l[j], u[j]).e1;
            if (ntok < kTok) {  // behind the sequence's end: the identity
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                    if (j >= ntok) l[j] = e1[j] = u[j] = both(0.f);
            }
            const float2 L = sum_by_pairs(l);
#pragma unroll
            for (int j = 0; j < kTok; ++j) S = advance(S, e1[j], u[j]);
#pragma unroll
            for (int j = kTok - 1; j >= 0; --j) {
                R = add(R, cotangent(j));  // 0 behind the end
                R = fma(e1[j], R, R);
            }
            sm.part[warp][lane] = make_float4(L.x, L.y, S.x, S.y);
            sm.rpart[warp][lane] = R;
        }
        arrive_warp(&sync.parts[0], lane);
        tc::mbar_wait(&sync.ready[0], k & 1, p.err);
        const float4 s = sm.part[warp][lane];
        float2 K = make_float2(s.z, s.w), dA = both(0.f);
        {
            // u[j] becomes the state before the token
            float2 h = make_float2(s.x, s.y);
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                const float2 before = h;
                h = advance(h, e1[j], u[j]);
                u[j] = before;
            }
        }
        int64_t o = t.base + (int64_t(warp * kTok + kTok - 1) * C + 2 * lane);
        const int c = t.ct * kGlrCols + 2 * lane;
        const bool a0 = c < C, a1 = c + 1 < C, even = C % 2 == 0;
        auto walk = [&](bool all) {
#pragma unroll
            for (int j = kTok - 1; j >= 0; --j, o -= C) {
                if (!all && j >= ntok) continue;
                const Sig sg = sigmoids(hd, gate(1, j), gate(2, j));
                const float2 sr = sg.sr, si = sg.si, er = sg.er, ei = sg.ei;
                const float2 w = square_minus_1(e1[j]);
                const float2 l = mul(A, sr), a = decay_of(l);
                const float2 rs = make_float2(inv_root(w.x), inv_root(w.y)), m = mul(make_float2(-w.x, -w.y), rs);
                const float2 six = mul(si, input(0, j));
                const float2 G = add(K, cotangent(j)), Gm = mul(G, m);
                // (G (h_t - s(i) x / m) would do, as a^2 + m^2 = 1, but for a small a it is
                // the difference of two numbers that are almost the same)
                const float2 as = mul(mul(a, six), rs);
                const float2 dl = mul(mul(G, a), add(u[j], make_float2(-as.x, -as.y)));
                dA = fma(dl, sr, dA);
                K = mul(a, G);
                store2<T, VEC>(p.dx + o, mul(Gm, si), all || a0, all || a1, even);
                store2<T, VEC>(p.di + o, mul(mul(Gm, six), mul(ei, si)), all || a0, all || a1, even);
                store2<T, VEC>(p.dr + o, mul(mul(dl, l), mul(er, sr)), all || a0, all || a1, even);
            }
        };
        if (t.full) walk(true);
        else walk(false);
        sm.dA[k & 1][warp][lane] = dA;
        if (warp == 0) sm.before[k & 1][lane] = K;
        __syncwarp();  // this warp's part of the stage is read
        load(k + NS);
        A = rates(k + 1);
    }
    arrive_warp(&sync.parts[0], lane);  // for the last tile's dA
}

// Column sums of a [rows, C] array: 32 columns a block, 32 rows at a time, each
// thread in order and then the 32 partial sums in order.  A thread of a long
// sequence adds thousands of terms of one sign, so it keeps what each addition
// rounds away (1e-4 of the sum without, 2^24 tokens).
__global__ void __launch_bounds__(1024)
row_sum_kernel(const float *__restrict__ part, int64_t rows, int C, float *__restrict__ out) {
    __shared__ float acc[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f, lost = 0.f;
    if (c < C)
#pragma unroll 4
        for (int64_t r = threadIdx.y; r < rows; r += 32) {
            const float v = __ldg(part + r * C + c), t = s + v, of_v = t - s;
            lost += (s - (t - of_v)) + (v - of_v);
            s = t;
        }
    acc[threadIdx.y][threadIdx.x] = isfinite(lost) ? s + lost : s;  // an infinite sum stays one
    __syncthreads();
    if (threadIdx.y == 0 && c < C) {
        float t = 0.f;
        for (int y = 0; y < 32; ++y) t += acc[y][threadIdx.x];
        out[c] = t;
    }
}

// the states of empty sequences
__global__ void __launch_bounds__(256)
copy_rows_kernel(const __grid_constant__ GlrRows rows, int C, const float *from, float *to) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= C) return;
    const int64_t o = int64_t(rows.id[blockIdx.y]) * C + c;
    to[o] = from ? from[o] : 0.f;
}

// ---------------------------------------------------------------------------
// decode step
// ---------------------------------------------------------------------------
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
glr_step_kernel(int batch, int C, const T *__restrict__ x, const T *__restrict__ r, const T *__restrict__ i,
                const float *__restrict__ A, float *__restrict__ state, T *__restrict__ y) {
    const int c = (blockIdx.x * 256 + threadIdx.x) * 2;
    const bool a0 = c < C, a1 = c + 1 < C;
    if (!a0) return;
    const float2 Av = load2<VEC>(A + c, a0, a1);
    const Held hd;
    for (int64_t b = blockIdx.y; b < batch; b += gridDim.y) {  // up to 2^31 - 1 rows: the next index may be past them
        const int64_t o = b * C + c;
        float2 xv, rv, iv, h;
        if (VEC) {
            xv = unpack2(x + o); rv = unpack2(r + o); iv = unpack2(i + o);
            h = *reinterpret_cast<const float2 *>(state + o);
        } else {
            const int64_t n = a1 ? o + 1 : o;
            xv = make_float2(to_f32<T>(x[o]), to_f32<T>(x[n]));
            rv = make_float2(to_f32<T>(r[o]), to_f32<T>(r[n]));
            iv = make_float2(to_f32<T>(i[o]), to_f32<T>(i[n]));
            h = make_float2(state[o], state[n]);
        }
        // one token after another goes on from what this leaves, so e^l - 1 where it is precise
        float2 l, u;
        const Decay d = token(hd, xv, at_least(rv), at_least(iv), Av, true, l, u);
        h = add(by_slope(l, mul(d.a, h), fma(d.e1, h, h)), u);
        store2<float, VEC>(state + o, h, a0, a1);
        store2<T, VEC>(y + o, h, a0, a1);
    }
}

// A persistent grid: one block an SM, or one a tile.
template <typename K, typename A>
cudaError_t launch_tiles(K kernel, int smem, const GlrShape &s, A &a, cudaStream_t stream) {
    const int64_t tiles = int64_t(s.nct) * s.nc * (s.nseq ? 1 : s.batch);
    const int64_t room = device_sm_count();
    a.tiles = int(tiles);
    a.dv = TileDivide{Divide::by(uint32_t(s.nct)), Divide::by(uint32_t(s.batch))};
    if (!smem_attr_once(reinterpret_cast<const void *>(kernel), smem)) return cudaErrorInvalidValue;
    kernel<<<unsigned(tiles < room ? tiles : room), kBlock, smem, stream>>>(a);
    return cudaGetLastError();
}

// Whether a tile's gates are formed ahead of the state of the one before it.  With
// few chains for the groups at work, the tiles of a chain wait for the sums of
// several groups, and those for their own states first.  With many, nothing waits
// long and the second stage of copies is worth more.  What counts are the chains that
// are in flight together: all of a batch's, whose tickets go round them chunk by
// chunk, but of packed sequences, which come one after another, the channel tiles
// of one, or as many sequences' as the groups hold at a time.  134 M values in
// bf16, us on the device ahead / not.  Batches: 16 chains 450 / 480, 32 289 / 338,
// 64 254 / 283, 128 238 / 248, 160 233 / 242, 256 224 / 230, 320 224 / 228, 640 222 / 220 (the
// border is on the safe side).  Packed, 2048 channels: 1 sequence 291 / 340, 16 299 /
// 374, 160 397 / 560; 5120: 16 258 / 283, 160 303 / 366; 10240: 16 239 / 244, 160 of 2
// chunks each 338 / 335.
bool hold_ahead(const GlrShape &s) {
    const int64_t groups = int64_t(device_sm_count()) * kGroups;
    int64_t chains = int64_t(s.nct) * (s.nseq ? s.nseq : s.batch);
    if (s.nseq) {
        const int64_t held = groups * s.nseq / s.nc;  // by the mean length
        const int64_t together = held > s.nct ? held : s.nct;
        if (together < chains) chains = together;
    }
    return 2 * chains <= groups;
}

template <typename T, bool VEC, bool PACK>
cudaError_t forward_typed(const GlrShape &s, const void *x, const void *r, const void *i, const float *A,
                          const float *h0, void *y, float *fin, float *states, const GlrPacked *packed,
                          const GlrScratch &ws, unsigned int *err, cudaStream_t stream) {
    FwdArgs<T> a;
    a.s = s; a.ws = ws;
    a.x = static_cast<const T *>(x); a.r = static_cast<const T *>(r); a.i = static_cast<const T *>(i);
    a.A = A; a.h0 = h0; a.y = static_cast<T *>(y); a.fin = fin; a.states = states;
    a.pk = packed ? *packed : GlrPacked{};
    a.err = err;
    if constexpr (VEC && sizeof(T) == 2)  // rows off the vectors have no registers left for it
        if (hold_ahead(s))
            return launch_tiles(glr_forward_kernel<T, VEC, PACK, true>, FwdPlan<T, true>::smem, s, a, stream);
    return launch_tiles(glr_forward_kernel<T, VEC, PACK, false>, FwdPlan<T, false>::smem, s, a, stream);
}

template <typename T, bool VEC, bool PACK>
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
    return launch_tiles(glr_backward_kernel<T, VEC, PACK>, BwdPlan<T, PACK>::smem, s, a, stream);
}

// rows of whole 16-byte vectors
bool vectors(int C, bool bf16) { return C % (bf16 ? 8 : 4) == 0; }

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
    return by_type(bf16, vectors(s.C, bf16), packed != nullptr, [&](auto t, auto even, auto pack) {
        return forward_typed<decltype(t), decltype(even)::value, decltype(pack)::value>(
            s, x, r, i, A, h0, y, fin, states, packed, ws, err, stream);
    });
}

cudaError_t launch_glr_backward(const GlrShape &s, bool bf16, const void *x, const void *r, const void *i,
                                const GlrPacked *packed, const float *A, const float *states, const void *dy,
                                const float *dfin, void *dx, void *dr, void *di, float *dinit, float *dA_part,
                                const GlrScratch &ws, unsigned int *err, cudaStream_t stream) {
    return by_type(bf16, s.C % 8 == 0, packed != nullptr, [&](auto t, auto even, auto pack) {
        return backward_typed<decltype(t), decltype(even)::value, decltype(pack)::value>(
            s, x, r, i, packed, A, states, dy, dfin, dx, dr, di, dinit, dA_part, ws, err, stream);
    });
}

cudaError_t launch_copy_rows(const GlrRows &rows, int C, const float *from, float *to, cudaStream_t stream) {
    copy_rows_kernel<<<dim3(unsigned((C + 255) / 256), unsigned(rows.n)), 256, 0, stream>>>(rows, C, from, to);
    return cudaGetLastError();
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
