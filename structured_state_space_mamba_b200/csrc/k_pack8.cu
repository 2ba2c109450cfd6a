// k_pack8.cu -- activations to 8-bit checkpoints and back (pack8.cuh has the
// format).
//
// HBM-bound: a value is 2 or 4 bytes read and 1 + 1/64 written, or the reverse
// (16384 x 5120: bf16 41 us to pack, 6.2 TB/s, 39 us to read back; fp32 60 and 64 us).
// Eight (bf16) or sixteen (fp32) lanes take a block of 64 values, one 16-byte vector
// a lane, and find its largest magnitude by shuffles; a thread has kUnroll
// blocks' loads in flight.  Rows that are no whole number of 8-value vectors go
// a warp a block with single-value accesses, eight blocks in flight (20000 x 1001
// bf16: 34 us, 1.8 TB/s).
#include "common.cuh"
#include "glr.h"
#include "pack8.cuh"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// values of a lane: one 16-byte vector
template <typename T> constexpr int kVals = 16 / sizeof(T);

__device__ __forceinline__ void load_vec(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load_vec(const float *p, float (&v)[4]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_vec(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
// the codes of a lane's values
__device__ __forceinline__ void store_codes(int8_t *p, const float (&v)[8], uint32_t ex) {
    *reinterpret_cast<uint2 *>(p) = pack8_eight(v, ex);
}
__device__ __forceinline__ void store_codes(int8_t *p, const float (&v)[4], uint32_t ex) {
    *reinterpret_cast<uint32_t *>(p) = pack8_four(v, ex);
}

// Where a lane's VALS values of its blocks lie: the first by a division, the next
// ones, kPer blocks on, by steps of whole rows and blocks of a row.  FLAT: whole
// blocks only, rows follow each other.
template <bool FLAT, int VALS>
struct Place {
    static constexpr int kLanes = kPackBlock / VALS, kPer = kThreads / kLanes;
    int64_t row, c, rows_on, blocks_on, nb, cols;
    int sub;
    __device__ __forceinline__ Place(int64_t n, int64_t nb_, int64_t cols_, int sub_)
        : nb(nb_), cols(cols_), sub(sub_) {
        if (FLAT) {
            row = n;
        } else {
            row = n / nb;
            c = n - row * nb;
            rows_on = kPer / nb;
            blocks_on = kPer - rows_on * nb;
        }
    }
    // the place; false behind the row's end
    __device__ __forceinline__ bool at(int64_t &o) const {
        if (FLAT) {
            o = row * kPackBlock + sub * VALS;
            return true;
        }
        const int64_t v = c * kPackBlock + sub * VALS;
        o = row * cols + v;
        return v < cols;
    }
    __device__ __forceinline__ void on() {
        if (FLAT) {
            row += kPer;
        } else {
            row += rows_on;
            c += blocks_on;
            if (c >= nb) {
                c -= nb;
                ++row;
            }
        }
    }
};

template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads)
pack8_kernel(int64_t blocks, int64_t nb, int64_t cols, const T *__restrict__ x, int8_t *__restrict__ codes,
             uint8_t *__restrict__ exps) {
    constexpr int V = kVals<T>;
    using P = Place<FLAT, V>;
    constexpr int kPer = P::kPer;  // blocks of one step
    const int sub = threadIdx.x % P::kLanes;
    const int64_t n0 = int64_t(blockIdx.x) * kPer * kUnroll + threadIdx.x / P::kLanes;
    float v[kUnroll][V];
    int64_t o[kUnroll];
    bool ok[kUnroll];
    P place(n0, nb, cols, sub);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k, place.on()) {
        const int64_t n = n0 + k * kPer;
        ok[k] = place.at(o[k]) && n < blocks;
        if (ok[k]) load_vec(x + o[k], v[k]);
        else
#pragma unroll
            for (int e = 0; e < V; ++e) v[k][e] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) m = max(m, __float_as_uint(v[k][e]) & 0x7fffffffu);
#pragma unroll
        for (int s = P::kLanes / 2; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
        if (!ok[k]) continue;
        const uint32_t ex = pack8_exp(m);
        store_codes(codes + o[k], v[k], ex);
        if (sub == 0) exps[n0 + k * kPer] = uint8_t(ex);
    }
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads)
unpack8_kernel(int64_t blocks, int64_t nb, int64_t cols, const int8_t *__restrict__ codes,
               const uint8_t *__restrict__ exps, T *__restrict__ out) {
    constexpr int V = kVals<T>;
    using P = Place<FLAT, V>;
    constexpr int kPer = P::kPer;
    const int sub = threadIdx.x % P::kLanes;
    const int64_t n0 = int64_t(blockIdx.x) * kPer * kUnroll + threadIdx.x / P::kLanes;
    uint32_t q[kUnroll][V / 4], ex[kUnroll];
    int64_t o[kUnroll];
    bool ok[kUnroll];
    P place(n0, nb, cols, sub);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k, place.on()) {
        const int64_t n = n0 + k * kPer;
        ok[k] = place.at(o[k]) && n < blocks;
        if (!ok[k]) continue;
        if constexpr (V == 8) {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(codes + o[k]));
            q[k][0] = w.x;
            q[k][1] = w.y;
        } else {
            q[k][0] = __ldg(reinterpret_cast<const uint32_t *>(codes + o[k]));
        }
        ex[k] = __ldg(exps + n);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        if (!ok[k]) continue;
        const float step = pack8_step(ex[k]);
        float v[V];
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 two = unpack8_two(q[k][e / 4] >> (8 * (e & 2)), step);
            v[e] = two.x;
            v[e + 1] = two.y;
        }
        store_vec(out + o[k], v);
    }
}

// any row length: a warp takes kRun blocks in a row, all of their loads on their way
// before the first is used, lanes at a stride of 32 values
constexpr int kRun = 8;
template <typename T>
__global__ void __launch_bounds__(kThreads)
pack8_any_kernel(int64_t blocks, int64_t nb, int64_t cols, const T *__restrict__ x, int8_t *__restrict__ codes,
                 uint8_t *__restrict__ exps) {
    const int lane = threadIdx.x & 31;
    const int64_t n0 = (int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kRun;
    if (n0 >= blocks) return;
    int64_t row = n0 / nb, c = (n0 - row * nb) * kPackBlock;
    float v[kRun][2];
    int64_t o[kRun];
    int left[kRun];  // values of the row from the block's first on, as far as they matter
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
        o[k] = row * cols + c + lane;
        left[k] = n0 + k < blocks ? int(min(cols - c, int64_t(kPackBlock))) : 0;
        v[k][0] = lane < left[k] ? to_f32<T>(x[o[k]]) : 0.f;
        v[k][1] = lane + 32 < left[k] ? to_f32<T>(x[o[k] + 32]) : 0.f;
        c += kPackBlock;
        if (c >= cols) {
            c = 0;
            ++row;
        }
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
        if (left[k] == 0) break;
        const uint32_t ex = pack8_exp(__reduce_max_sync(
            0xffffffffu, max(__float_as_uint(v[k][0]) & 0x7fffffffu, __float_as_uint(v[k][1]) & 0x7fffffffu)));
        const float inv = pack8_inv(ex);
        const bool edge = ex >= kPackEdge;  // the same for the whole warp
        const uint32_t a = edge ? uint32_t(pack8_code(v[k][0], inv)) : pack8_fast(v[k][0], inv);
        const uint32_t b = edge ? uint32_t(pack8_code(v[k][1], inv)) : pack8_fast(v[k][1], inv);
        if (lane < left[k]) codes[o[k]] = int8_t(a);
        if (lane + 32 < left[k]) codes[o[k] + 32] = int8_t(b);
        if (lane == 0) exps[n0 + k] = uint8_t(ex);
    }
}
template <typename T>
__global__ void __launch_bounds__(kThreads)
unpack8_any_kernel(int64_t blocks, int64_t nb, int64_t cols, const int8_t *__restrict__ codes,
                   const uint8_t *__restrict__ exps, T *__restrict__ out) {
    const int lane = threadIdx.x & 31;
    const int64_t n0 = (int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kRun;
    if (n0 >= blocks) return;
    int64_t row = n0 / nb, c = (n0 - row * nb) * kPackBlock;
    int8_t q[kRun][2];
    uint32_t ex[kRun];
    int64_t o[kRun];
    int left[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
        o[k] = row * cols + c + lane;
        left[k] = n0 + k < blocks ? int(min(cols - c, int64_t(kPackBlock))) : 0;
        q[k][0] = lane < left[k] ? codes[o[k]] : int8_t(0);
        q[k][1] = lane + 32 < left[k] ? codes[o[k] + 32] : int8_t(0);
        ex[k] = left[k] ? exps[n0 + k] : 1u;
        c += kPackBlock;
        if (c >= cols) {
            c = 0;
            ++row;
        }
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
        const float step = pack8_step(ex[k]);
        if (lane < left[k]) out[o[k]] = from_f32<T>(float(q[k][0]) * step);
        if (lane + 32 < left[k]) out[o[k] + 32] = from_f32<T>(float(q[k][1]) * step);
    }
}

struct Plan {
    int64_t nb, blocks;
    unsigned vec_grid, any_grid;
    bool fits;
};
template <typename T>
Plan plan_of(int64_t rows, int64_t cols) {
    Plan p;
    p.nb = (cols + kPackBlock - 1) / kPackBlock;
    p.blocks = rows * p.nb;
    const int64_t per = Place<true, kVals<T>>::kPer * kUnroll, any = kThreads / 32 * kRun;
    const int64_t g = (p.blocks + per - 1) / per, h = (p.blocks + any - 1) / any;
    p.fits = g <= 0x7fffffff && h <= 0x7fffffff;
    p.vec_grid = unsigned(g);
    p.any_grid = unsigned(h);
    return p;
}

template <typename T>
cudaError_t pack_typed(int64_t rows, int64_t cols, const T *x, int8_t *codes, uint8_t *exps, cudaStream_t st) {
    const Plan p = plan_of<T>(rows, cols);
    if (!p.fits) return cudaErrorInvalidValue;
    if (cols % kPackBlock == 0)
        pack8_kernel<T, true><<<p.vec_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, x, codes, exps);
    else if (cols % kVals<T> == 0)
        pack8_kernel<T, false><<<p.vec_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, x, codes, exps);
    else
        pack8_any_kernel<T><<<p.any_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, x, codes, exps);
    return cudaGetLastError();
}
template <typename T>
cudaError_t unpack_typed(int64_t rows, int64_t cols, const int8_t *codes, const uint8_t *exps, T *out,
                         cudaStream_t st) {
    const Plan p = plan_of<T>(rows, cols);
    if (!p.fits) return cudaErrorInvalidValue;
    if (cols % kPackBlock == 0)
        unpack8_kernel<T, true><<<p.vec_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, codes, exps, out);
    else if (cols % kVals<T> == 0)
        unpack8_kernel<T, false><<<p.vec_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, codes, exps, out);
    else
        unpack8_any_kernel<T><<<p.any_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, codes, exps, out);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pack8(int64_t rows, int64_t cols, bool bf16, const void *x, int8_t *codes, uint8_t *exps,
                         cudaStream_t stream) {
    return bf16 ? pack_typed(rows, cols, static_cast<const __nv_bfloat16 *>(x), codes, exps, stream)
                : pack_typed(rows, cols, static_cast<const float *>(x), codes, exps, stream);
}

cudaError_t launch_unpack8(int64_t rows, int64_t cols, bool bf16, const int8_t *codes, const uint8_t *exps,
                           void *out, cudaStream_t stream) {
    return bf16 ? unpack_typed(rows, cols, codes, exps, static_cast<__nv_bfloat16 *>(out), stream)
                : unpack_typed(rows, cols, codes, exps, static_cast<float *>(out), stream);
}

}  // namespace ssd
