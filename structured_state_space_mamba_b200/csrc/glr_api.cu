// glr_api.cu -- the C ABI of the gated linear recurrence, of the 8-bit
// checkpoints and of the norm and rotation of B and C (declared in
// include/ssd.h): argument checks, scratch and launches.  Every error is
// detected before the first launch.
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/ssd.h"
#include "glr.h"
#include "norm_rotate.h"

namespace {

using ssd::GlrPacked;
using ssd::GlrScratch;
using ssd::GlrShape;

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool misaligned(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

ssd_status_t check_glr_dims(const ssd_glr_dims_t *dims) {
    if (!dims) return SSD_ERR_NULL_ARG;
    const ssd_glr_dims_t &a = *dims;
    if (a.batch <= 0 || a.seqlen <= 0 || a.channels <= 0 || a.reserved != 0) return SSD_ERR_INVALID_DIM;
    if (a.dtype != SSD_F32 && a.dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (a.seqlen > (int64_t(1) << 30) || a.channels > (int64_t(1) << 24) || a.batch > 0x7fffffff)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Chunks of every sequence, in all; checks the offsets.
ssd_status_t count_chunks(const ssd_glr_dims_t &a, const int64_t *cu, int64_t nseq, int64_t *chunks) {
    int64_t n = 0;
    if (!cu) {
        n = ceil_div(a.seqlen, ssd::kGlrChunk);
        if (n > 0x7fffffff / a.batch) return SSD_ERR_UNSUPPORTED;
        n *= a.batch;
    } else {
        if (a.batch != 1 || nseq <= 0 || cu[0] != 0 || cu[nseq] != a.seqlen) return SSD_ERR_INVALID_DIM;
        if (nseq > 0x7fffffff) return SSD_ERR_UNSUPPORTED;
        for (int64_t j = 0; j < nseq; ++j)
            if (cu[j + 1] < cu[j] || cu[j + 1] > a.seqlen) return SSD_ERR_INVALID_DIM;
        for (int64_t j = 0; j < nseq; ++j) n += ceil_div(cu[j + 1] - cu[j], ssd::kGlrChunk);
    }
    if (n > 0x7fffffff / ceil_div(a.channels, ssd::kGlrCols)) return SSD_ERR_UNSUPPORTED;
    *chunks = n;
    return SSD_OK;
}

// The launches of one call: the whole batch, or the sequences that are not empty
// in groups.  next() fills `s`, with true while there is one.
struct Groups {
    const ssd_glr_dims_t &a;
    const int64_t *cu;
    int64_t nseq;
    int64_t at = 0, chunk = 0;
    bool next(GlrShape &s, bool &linked) {
        std::memset(&s, 0, sizeof(s));
        s.C = int(a.channels);
        s.T = int(a.seqlen);
        s.nct = int(ceil_div(a.channels, ssd::kGlrCols));
        if (!cu) {
            if (at) return false;
            at = 1;
            s.batch = int(a.batch);
            s.nc = int(ceil_div(a.seqlen, ssd::kGlrChunk));
            linked = s.nc > 1;
            return true;
        }
        s.batch = 1;
        s.chunk0 = chunk;
        linked = false;
        for (; at < nseq && s.nseq < ssd::kGlrSeqs; ++at) {
            const int64_t len = cu[at + 1] - cu[at];
            if (len == 0) continue;
            s.id[s.nseq] = int(at);
            s.start[s.nseq] = int(cu[at]);
            s.len[s.nseq] = int(len);
            s.cb[s.nseq] = s.nc;
            const int n = int(ceil_div(len, ssd::kGlrChunk));
            linked |= n > 1;
            s.nc += n;
            ++s.nseq;
        }
        s.cb[s.nseq] = s.nc;
        chunk += s.nc;
        return s.nseq > 0;
    }
};

// Scratch of the launches, one after another inside an allocation.
struct ScratchPlan {
    size_t bytes = 0;  // so far
    static size_t tiles(const GlrShape &s) { return size_t(s.nct) * s.nc * (s.nseq ? 1 : s.batch); }
    // adds a launch; its scratch, when the allocation is there
    GlrScratch add(const GlrShape &s, bool linked, char *buf = nullptr) {
        GlrScratch w = {};
        if (!linked) return w;
        if (buf) {
            w.ticket = reinterpret_cast<unsigned int *>(buf + bytes);
            w.sums = reinterpret_cast<float4 *>(buf + bytes + kAlign);
            w.state = reinterpret_cast<float2 *>(w.sums + tiles(s) * 32);
        }
        bytes += kAlign + align_up(tiles(s) * 32 * (sizeof(float4) + sizeof(float2)));
        return w;
    }
};

// An empty sequence leaves its state as it came.
ssd_status_t copy_empty(const int64_t *cu, int64_t nseq, int64_t C, const float *from, float *to, cudaStream_t st) {
    if (!cu || !to) return SSD_OK;
    ssd::GlrRows rows;
    rows.n = 0;
    for (int64_t j = 0; j <= nseq; ++j) {
        if (j < nseq && cu[j + 1] == cu[j]) rows.id[rows.n++] = int(j);
        if (rows.n == ssd::kGlrRows || (j == nseq && rows.n > 0)) {
            if (ssd::launch_copy_rows(rows, int(C), from, to, st) != cudaSuccess) return SSD_ERR_CUDA;
            rows.n = 0;
        }
    }
    return SSD_OK;
}

ssd_status_t take_packed(const ssd_packed8_t *in, GlrPacked *out) {
    for (int n = 0; n < 3; ++n) {
        if (!in[n].codes || !in[n].exps) return SSD_ERR_NULL_ARG;
        if (misaligned(in[n].codes) || misaligned(in[n].exps)) return SSD_ERR_MISALIGNED;
        out->codes[n] = in[n].codes;
        out->exps[n] = in[n].exps;
    }
    return SSD_OK;
}

ssd_status_t check_pack(int64_t rows, int64_t cols, int dtype, const void *p, const ssd_packed8_t *packed) {
    if (!p || !packed || !packed->codes || !packed->exps) return SSD_ERR_NULL_ARG;
    if (rows <= 0 || cols <= 0) return SSD_ERR_INVALID_DIM;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (ceil_div(cols, SSD_PACK8_BLOCK) > (int64_t(1) << 33) / rows) return SSD_ERR_UNSUPPORTED;
    if (misaligned(p) || misaligned(packed->codes) || misaligned(packed->exps)) return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

ssd_status_t rotate_shape(const ssd_rotate_dims_t *dims, ssd::RotateShape *s) {
    if (!dims) return SSD_ERR_NULL_ARG;
    const ssd_rotate_dims_t &a = *dims;
    if (a.batch <= 0 || a.seqlen <= 0 || a.ngroups <= 0 || a.dstate <= 0 || a.reserved != 0 || a.rotary < 0 ||
        a.rotary > a.dstate || a.rotary % 2 != 0 || !(a.eps > 0.f))
        return SSD_ERR_INVALID_DIM;
    if (a.dtype != SSD_F32 && a.dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (a.dstate > 256 || a.batch > 0x7fffffff / a.seqlen || a.ngroups > (1 << 20)) return SSD_ERR_UNSUPPORTED;
    s->tokens = a.batch * a.seqlen;
    s->B_batch = a.B_batch_stride; s->B_token = a.B_token_stride;
    s->C_batch = a.C_batch_stride; s->C_token = a.C_token_stride;
    s->T = int(a.seqlen); s->G = int(a.ngroups); s->N = int(a.dstate); s->rotary = int(a.rotary);
    s->lanes = 4;
    while (s->lanes * 8 < s->N) s->lanes *= 2;
    s->interleaved = a.interleaved ? 1 : 0;
    s->eps = a.eps;
    return SSD_OK;
}

bool off(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
// what a norm and rotation reads: whole tensors on 16 bytes, the rest by elements
bool off_rotate(const ssd_rotate_dims_t &a, const void *Bm, const void *Cm, const int64_t *positions,
                const float *inv_freq, const float *weight_B, const float *weight_C) {
    const uintptr_t es = a.dtype == SSD_BF16 ? 2 : 4;
    return off(Bm, es) || off(Cm, es) || off(positions, 8) || off(inv_freq, 4) || off(weight_B, 4) || off(weight_C, 4);
}

}  // namespace

extern "C" {

int64_t ssd_glr_chunk_rows(const ssd_glr_dims_t *dims, const int64_t *cu_seqlens, int64_t nseq) {
    int64_t chunks = 0;
    if (check_glr_dims(dims) != SSD_OK || count_chunks(*dims, cu_seqlens, nseq, &chunks) != SSD_OK) return 0;
    return chunks;
}

ssd_status_t ssd_glr_forward(const ssd_glr_dims_t *dims, const int64_t *cu_seqlens, int64_t nseq, const void *x,
                             const void *r, const void *i, const float *A, const float *init_state, void *y_out,
                             float *final_state_out, float *chunk_states_out, const ssd_packed8_t *packed_out,
                             void *stream) {
    ssd_status_t s = check_glr_dims(dims);
    if (s != SSD_OK) return s;
    int64_t chunks = 0;
    s = count_chunks(*dims, cu_seqlens, nseq, &chunks);
    if (s != SSD_OK) return s;
    if (!x || !r || !i || !A || !y_out) return SSD_ERR_NULL_ARG;
    const void *ptrs[] = {x, r, i, A, init_state, y_out, final_state_out, chunk_states_out};
    for (const void *p : ptrs)
        if (misaligned(p)) return SSD_ERR_MISALIGNED;
    GlrPacked pk = {};
    if (packed_out && (s = take_packed(packed_out, &pk)) != SSD_OK) return s;
    unsigned int *err = ssd::device_error_word();
    if (!err) return SSD_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf16 = dims->dtype == SSD_BF16;

    GlrShape shape;
    bool linked = false;
    ScratchPlan plan;
    for (Groups g{*dims, cu_seqlens, nseq}; g.next(shape, linked);) plan.add(shape, linked);
    char *buf = nullptr;
    if (plan.bytes) {
        if (ssd::workspace_alloc(reinterpret_cast<void **>(&buf), plan.bytes, st) != cudaSuccess) {
            cudaGetLastError();
            return SSD_ERR_WORKSPACE;
        }
        if (cudaMemsetAsync(buf, 0xff, plan.bytes, st) != cudaSuccess) s = SSD_ERR_CUDA;
    }
    ScratchPlan used;
    for (Groups g{*dims, cu_seqlens, nseq}; s == SSD_OK && g.next(shape, linked);)
        if (ssd::launch_glr_forward(shape, bf16, x, r, i, A, init_state, y_out, final_state_out, chunk_states_out,
                                    packed_out ? &pk : nullptr, used.add(shape, linked, buf), err,
                                    st) != cudaSuccess)
            s = SSD_ERR_CUDA;
    if (s == SSD_OK) s = copy_empty(cu_seqlens, nseq, dims->channels, init_state, final_state_out, st);
    if (buf && cudaFreeAsync(buf, st) != cudaSuccess && s == SSD_OK) s = SSD_ERR_CUDA;
    return s;
}

ssd_status_t ssd_glr_backward(const ssd_glr_dims_t *dims, const int64_t *cu_seqlens, int64_t nseq, const void *x,
                              const void *r, const void *i, const ssd_packed8_t *packed, const float *A,
                              const float *chunk_states, const void *dy, const float *dfinal_state, void *dx,
                              void *dr, void *di, float *dA, float *dinit_state, void *stream) {
    ssd_status_t s = check_glr_dims(dims);
    if (s != SSD_OK) return s;
    int64_t chunks = 0;
    s = count_chunks(*dims, cu_seqlens, nseq, &chunks);
    if (s != SSD_OK) return s;
    if (!A || !chunk_states || !dy || !dx || !dr || !di || !dA) return SSD_ERR_NULL_ARG;
    if (!packed && (!x || !r || !i)) return SSD_ERR_NULL_ARG;
    if (packed && (x || r || i)) return SSD_ERR_INVALID_DIM;
    const void *ptrs[] = {x, r, i, A, chunk_states, dy, dfinal_state, dx, dr, di, dA, dinit_state};
    for (const void *p : ptrs)
        if (misaligned(p)) return SSD_ERR_MISALIGNED;
    GlrPacked pk = {};
    if (packed && (s = take_packed(packed, &pk)) != SSD_OK) return s;
    unsigned int *err = ssd::device_error_word();
    if (!err) return SSD_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf16 = dims->dtype == SSD_BF16;
    const int C = int(dims->channels);

    GlrShape shape;
    bool linked = false;
    ScratchPlan plan;
    for (Groups g{*dims, cu_seqlens, nseq}; g.next(shape, linked);) plan.add(shape, linked);
    char *buf = nullptr;
    const size_t part_off = plan.bytes, bytes = part_off + size_t(chunks) * C * sizeof(float);
    if (ssd::workspace_alloc(reinterpret_cast<void **>(&buf), bytes, st) != cudaSuccess) {
        cudaGetLastError();
        return SSD_ERR_WORKSPACE;
    }
    float *part = reinterpret_cast<float *>(buf + part_off);
    if (plan.bytes && cudaMemsetAsync(buf, 0xff, plan.bytes, st) != cudaSuccess) s = SSD_ERR_CUDA;
    ScratchPlan used;
    for (Groups g{*dims, cu_seqlens, nseq}; s == SSD_OK && g.next(shape, linked);)
        if (ssd::launch_glr_backward(shape, bf16, x, r, i, packed ? &pk : nullptr, A, chunk_states, dy, dfinal_state,
                                     dx, dr, di, dinit_state, part, used.add(shape, linked, buf), err,
                                     st) != cudaSuccess)
            s = SSD_ERR_CUDA;
    if (s == SSD_OK && ssd::launch_row_sum(part, chunks, C, dA, st) != cudaSuccess) s = SSD_ERR_CUDA;
    if (s == SSD_OK) s = copy_empty(cu_seqlens, nseq, dims->channels, dfinal_state, dinit_state, st);
    if (cudaFreeAsync(buf, st) != cudaSuccess && s == SSD_OK) s = SSD_ERR_CUDA;
    return s;
}

ssd_status_t ssd_glr_step(const ssd_glr_dims_t *dims, const void *x_t, const void *r_t, const void *i_t,
                          const float *A, float *state, void *y_t, void *stream) {
    const ssd_status_t s = check_glr_dims(dims);
    if (s != SSD_OK) return s;
    if (dims->seqlen != 1) return SSD_ERR_INVALID_DIM;
    if (!x_t || !r_t || !i_t || !A || !state || !y_t) return SSD_ERR_NULL_ARG;
    const void *ptrs[] = {x_t, r_t, i_t, A, state, y_t};
    for (const void *p : ptrs)
        if (misaligned(p)) return SSD_ERR_MISALIGNED;
    return ssd::launch_glr_step(int(dims->batch), int(dims->channels), dims->dtype == SSD_BF16, x_t, r_t, i_t, A,
                                state, y_t, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SSD_OK
               : SSD_ERR_CUDA;
}

ssd_status_t ssd_pack8(int64_t rows, int64_t cols, int dtype, const void *x, const ssd_packed8_t *packed,
                       void *stream) {
    const ssd_status_t s = check_pack(rows, cols, dtype, x, packed);
    if (s != SSD_OK) return s;
    return ssd::launch_pack8(rows, cols, dtype == SSD_BF16, x, packed->codes, packed->exps,
                             static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SSD_OK
               : SSD_ERR_CUDA;
}

ssd_status_t ssd_unpack8(int64_t rows, int64_t cols, int dtype, const ssd_packed8_t *packed, void *out,
                         void *stream) {
    const ssd_status_t s = check_pack(rows, cols, dtype, out, packed);
    if (s != SSD_OK) return s;
    return ssd::launch_unpack8(rows, cols, dtype == SSD_BF16, packed->codes, packed->exps, out,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SSD_OK
               : SSD_ERR_CUDA;
}

ssd_status_t ssd_norm_rotate(const ssd_rotate_dims_t *dims, const void *Bm, const void *Cm,
                             const int64_t *positions, const float *inv_freq, const float *weight_B,
                             const float *weight_C, void *B_out, void *C_out, void *stream) {
    ssd::RotateShape sh;
    const ssd_status_t s = rotate_shape(dims, &sh);
    if (s != SSD_OK) return s;
    if (!Bm || !Cm || !positions || (!inv_freq && sh.rotary) || !B_out || !C_out) return SSD_ERR_NULL_ARG;
    if (misaligned(B_out) || misaligned(C_out) ||
        off_rotate(*dims, Bm, Cm, positions, inv_freq, weight_B, weight_C))
        return SSD_ERR_MISALIGNED;
    return ssd::launch_norm_rotate(sh, dims->dtype == SSD_BF16, Bm, Cm, positions, inv_freq, weight_B, weight_C,
                                   B_out, C_out, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SSD_OK
               : SSD_ERR_CUDA;
}

ssd_status_t ssd_norm_rotate_backward(const ssd_rotate_dims_t *dims, const void *dB_out, const void *dC_out,
                                      const void *Bm, const void *Cm, const int64_t *positions,
                                      const float *inv_freq, const float *weight_B, const float *weight_C, void *dB,
                                      void *dC, float *dweight_B, float *dweight_C, void *stream) {
    ssd::RotateShape sh;
    ssd_status_t s = rotate_shape(dims, &sh);
    if (s != SSD_OK) return s;
    if (!dB_out || !dC_out || !Bm || !Cm || !positions || (!inv_freq && sh.rotary) || !dB || !dC)
        return SSD_ERR_NULL_ARG;
    const void *ptrs[] = {dB_out, dC_out, dB, dC};
    for (const void *p : ptrs)
        if (misaligned(p)) return SSD_ERR_MISALIGNED;
    if (off_rotate(*dims, Bm, Cm, positions, inv_freq, weight_B, weight_C) || off(dweight_B, 4) || off(dweight_C, 4))
        return SSD_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *part = nullptr;
    if (dweight_B || dweight_C) {
        const size_t bytes = size_t(ssd::norm_rotate_backward_blocks(sh)) * 2 * sh.N * sizeof(float);
        if (ssd::workspace_alloc(reinterpret_cast<void **>(&part), bytes, st) != cudaSuccess) {
            cudaGetLastError();
            return SSD_ERR_WORKSPACE;
        }
    }
    if (ssd::launch_norm_rotate_backward(sh, dims->dtype == SSD_BF16, dB_out, dC_out, Bm, Cm, positions, inv_freq,
                                         weight_B, weight_C, dB, dC, part, dweight_B, dweight_C, st) != cudaSuccess)
        s = SSD_ERR_CUDA;
    if (part && cudaFreeAsync(part, st) != cudaSuccess && s == SSD_OK) s = SSD_ERR_CUDA;
    return s;
}

}  // extern "C"
