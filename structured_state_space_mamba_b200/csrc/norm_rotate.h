// norm_rotate.h -- host-side launchers of the norm and rotation of B and C
// (internal to libssd.so).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

struct RotateShape {
    int64_t tokens;                    // batch * T
    int64_t B_batch, B_token, C_batch, C_token;  // strides in elements
    int T, G, N, rotary;
    int lanes;                         // lanes of a token: N / 8, up to a power of two, 4 to 32
    int interleaved;
    float eps;
};

cudaError_t launch_norm_rotate(const RotateShape &s, bool bf16, const void *Bm, const void *Cm,
                               const int64_t *positions, const float *inv_freq, const float *wB, const float *wC,
                               void *Bo, void *Co, cudaStream_t stream);
// part: fp32 [norm_rotate_backward_blocks][2][N], or nullptr (no weight gradients)
int norm_rotate_backward_blocks(const RotateShape &s);
cudaError_t launch_norm_rotate_backward(const RotateShape &s, bool bf16, const void *dBo, const void *dCo,
                                        const void *Bm, const void *Cm, const int64_t *positions,
                                        const float *inv_freq, const float *wB, const float *wC, void *dB, void *dC,
                                        float *part, float *dwB, float *dwC, cudaStream_t stream);

}  // namespace ssd
