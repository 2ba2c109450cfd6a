// glr.h -- host-side launchers of the gated linear recurrence and of the 8-bit
// checkpoints (internal to libssd.so).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssd.h"

namespace ssd {

constexpr int kGlrChunk = SSD_GLR_CHUNK;  // tokens of a tile
constexpr int kGlrCols = 64;              // channels of a tile (one checkpoint block)
// packed sequences of one launch: their offsets travel as kernel parameters
// (4 KB), so a captured launch holds them and no copy of the caller's host
// array is in flight
constexpr int kGlrSeqs = 160;

struct GlrShape {
    int batch, T, C;   // T: tokens of a row (of all sequences when they are packed)
    int nct;           // channel tiles
    int nc;            // chunks of a row; of all this launch's sequences when packed
    int nseq;          // packed sequences of this launch, 0 for a batch
    int64_t chunk0;    // row of chunk_states of this launch's first chunk
    int id[kGlrSeqs];          // row of the states
    int start[kGlrSeqs];       // first token
    int len[kGlrSeqs];         // tokens, at least 1
    int cb[kGlrSeqs + 1];      // chunks before the sequence
};

// Scratch of one launch: the hand-off of the states between the tiles of a
// chain, all ones at the start.  With one chunk a sequence there is none and
// every pointer is null.
struct GlrScratch {
    unsigned int *ticket;  // the last tile taken
    float4 *sums;          // [tiles][32] decays and sums of two channels a lane
    float2 *state;         // [tiles][32] the state that leaves the tile
};

struct GlrPacked {
    int8_t *codes[3];
    uint8_t *exps[3];
};

cudaError_t launch_glr_forward(const GlrShape &s, bool bf16, const void *x, const void *r, const void *i,
                               const float *A, const float *h0, void *y, float *fin, float *states,
                               const GlrPacked *packed, const GlrScratch &ws, unsigned int *err,
                               cudaStream_t stream);
cudaError_t launch_glr_backward(const GlrShape &s, bool bf16, const void *x, const void *r, const void *i,
                                const GlrPacked *packed, const float *A, const float *states, const void *dy,
                                const float *dfin, void *dx, void *dr, void *di, float *dinit, float *dA_part,
                                const GlrScratch &ws, unsigned int *err, cudaStream_t stream);
// rows id[0 .. n) of `to` [., C] from those of `from`, or zeros without it
constexpr int kGlrRows = 512;
struct GlrRows {
    int n;
    int id[kGlrRows];
};
cudaError_t launch_copy_rows(const GlrRows &rows, int C, const float *from, float *to, cudaStream_t stream);
// dA[c] = sum of the rows of part [rows, C], in a fixed order
cudaError_t launch_row_sum(const float *part, int64_t rows, int C, float *out, cudaStream_t stream);
cudaError_t launch_glr_step(int batch, int C, bool bf16, const void *x, const void *r, const void *i,
                            const float *A, float *state, void *y, cudaStream_t stream);

cudaError_t launch_pack8(int64_t rows, int64_t cols, bool bf16, const void *x, int8_t *codes, uint8_t *exps,
                         cudaStream_t stream);
cudaError_t launch_unpack8(int64_t rows, int64_t cols, bool bf16, const int8_t *codes, const uint8_t *exps,
                           void *out, cudaStream_t stream);

// shared with the other entry points (ssd_api.cu)
unsigned int *device_error_word();
cudaError_t workspace_alloc(void **p, size_t bytes, cudaStream_t st);

}  // namespace ssd
