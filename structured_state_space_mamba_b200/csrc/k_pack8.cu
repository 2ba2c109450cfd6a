// k_pack8.cu -- activations to 8-bit checkpoints and back (pack8.cuh has the
// format).
//
// HBM-bound: a value is 2 or 4 bytes read and 1 + 1/64 written, or the reverse.
// Eight lanes take a block of 64 values, 16 or 32 bytes a lane in one or two
// vectors, and find its largest magnitude by shuffles; a thread has kUnroll
// blocks' loads in flight.  Rows that are no whole number of 8-value vectors go
// one warp a block with single-value accesses.
#include "common.cuh"
#include "glr.h"
#include "pack8.cuh"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Where a lane's eight values of block n lie (n = row * nb + block of the row);
// false behind the row's end.  FLAT: whole blocks only, rows follow each other.
template <bool FLAT>
__device__ __forceinline__ bool place(int64_t n, int64_t nb, int64_t cols, int sub, int64_t &o) {
    if (FLAT) {
        o = n * kPackBlock + sub * 8;
        return true;
    }
    const int64_t row = n / nb, c = (n - row * nb) * kPackBlock + sub * 8;
    o = row * cols + c;
    return c < cols;
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads)
pack8_kernel(int64_t blocks, int64_t nb, int64_t cols, const T *__restrict__ x, int8_t *__restrict__ codes,
             uint8_t *__restrict__ exps) {
    constexpr int kPer = kThreads / 8;  // blocks of one step
    const int sub = threadIdx.x & 7;
    const int64_t n0 = int64_t(blockIdx.x) * kPer * kUnroll + (threadIdx.x >> 3);
    float v[kUnroll][8];
    int64_t o[kUnroll];
    bool ok[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        const int64_t n = n0 + k * kPer;
        ok[k] = n < blocks && place<FLAT>(n, nb, cols, sub, o[k]);
        if (ok[k]) load8(x + o[k], v[k]);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[k][e]) & 0x7fffffffu);
#pragma unroll
        for (int s = 4; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
        if (!ok[k]) continue;
        const uint32_t ex = pack8_exp(m);
        *reinterpret_cast<uint2 *>(codes + o[k]) = pack8_eight(v[k], ex);
        if (sub == 0) exps[n0 + k * kPer] = uint8_t(ex);
    }
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads)
unpack8_kernel(int64_t blocks, int64_t nb, int64_t cols, const int8_t *__restrict__ codes,
               const uint8_t *__restrict__ exps, T *__restrict__ out) {
    constexpr int kPer = kThreads / 8;
    const int sub = threadIdx.x & 7;
    const int64_t n0 = int64_t(blockIdx.x) * kPer * kUnroll + (threadIdx.x >> 3);
    uint2 q[kUnroll];
    uint32_t ex[kUnroll];
    int64_t o[kUnroll];
    bool ok[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        const int64_t n = n0 + k * kPer;
        ok[k] = n < blocks && place<FLAT>(n, nb, cols, sub, o[k]);
        if (!ok[k]) continue;
        q[k] = __ldg(reinterpret_cast<const uint2 *>(codes + o[k]));
        ex[k] = __ldg(exps + n);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        if (!ok[k]) continue;
        const float step = pack8_step(ex[k]);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 two = unpack8_two((e < 4 ? q[k].x : q[k].y) >> (8 * (e & 2)), step);
            v[e] = two.x;
            v[e + 1] = two.y;
        }
        store8(out + o[k], v);
    }
}

// any row length: one warp a block, lanes at a stride of 32 values
template <typename T>
__global__ void __launch_bounds__(kThreads)
pack8_any_kernel(int64_t blocks, int64_t nb, int64_t cols, const T *__restrict__ x, int8_t *__restrict__ codes,
                 uint8_t *__restrict__ exps) {
    const int lane = threadIdx.x & 31;
    const int64_t n = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (n >= blocks) return;
    const int64_t row = n / nb, c = (n - row * nb) * kPackBlock + lane, o = row * cols + c;
    const bool a = c < cols, b = c + 32 < cols;
    const float v = a ? to_f32<T>(x[o]) : 0.f, w = b ? to_f32<T>(x[o + 32]) : 0.f;
    const uint32_t m = __reduce_max_sync(0xffffffffu, max(__float_as_uint(v) & 0x7fffffffu,
                                                          __float_as_uint(w) & 0x7fffffffu));
    const uint32_t ex = pack8_exp(m);
    const float inv = pack8_inv(ex);
    if (a) codes[o] = int8_t(pack8_code(v, inv));
    if (b) codes[o + 32] = int8_t(pack8_code(w, inv));
    if (lane == 0) exps[n] = uint8_t(ex);
}
template <typename T>
__global__ void __launch_bounds__(kThreads)
unpack8_any_kernel(int64_t blocks, int64_t nb, int64_t cols, const int8_t *__restrict__ codes,
                   const uint8_t *__restrict__ exps, T *__restrict__ out) {
    const int lane = threadIdx.x & 31;
    const int64_t n = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (n >= blocks) return;
    const int64_t row = n / nb, c = (n - row * nb) * kPackBlock + lane, o = row * cols + c;
    const float step = pack8_step(exps[n]);
    if (c < cols) out[o] = from_f32<T>(float(codes[o]) * step);
    if (c + 32 < cols) out[o + 32] = from_f32<T>(float(codes[o + 32]) * step);
}

struct Plan {
    int64_t nb, blocks;
    unsigned vec_grid, any_grid;
    bool fits;
};
Plan plan_of(int64_t rows, int64_t cols) {
    Plan p;
    p.nb = (cols + kPackBlock - 1) / kPackBlock;
    p.blocks = rows * p.nb;
    const int64_t per = kThreads / 8 * kUnroll, any = kThreads / 32;
    const int64_t g = (p.blocks + per - 1) / per, h = (p.blocks + any - 1) / any;
    p.fits = h <= 0x7fffffff;
    p.vec_grid = unsigned(g);
    p.any_grid = unsigned(h);
    return p;
}

template <typename T>
cudaError_t pack_typed(int64_t rows, int64_t cols, const T *x, int8_t *codes, uint8_t *exps, cudaStream_t st) {
    const Plan p = plan_of(rows, cols);
    if (!p.fits) return cudaErrorInvalidValue;
    if (cols % kPackBlock == 0)
        pack8_kernel<T, true><<<p.vec_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, x, codes, exps);
    else if (cols % 8 == 0)
        pack8_kernel<T, false><<<p.vec_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, x, codes, exps);
    else
        pack8_any_kernel<T><<<p.any_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, x, codes, exps);
    return cudaGetLastError();
}
template <typename T>
cudaError_t unpack_typed(int64_t rows, int64_t cols, const int8_t *codes, const uint8_t *exps, T *out,
                         cudaStream_t st) {
    const Plan p = plan_of(rows, cols);
    if (!p.fits) return cudaErrorInvalidValue;
    if (cols % kPackBlock == 0)
        unpack8_kernel<T, true><<<p.vec_grid, kThreads, 0, st>>>(p.blocks, p.nb, cols, codes, exps, out);
    else if (cols % 8 == 0)
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
