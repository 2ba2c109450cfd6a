"""ctypes binding of ``libssd.so`` (the C ABI in ``include/ssd.h``).

Argument marshalling only: shapes, dtypes and devices of torch tensors are
checked, their device pointers and the current CUDA stream are passed to the C
call, and a non-zero status is raised as :class:`SSDError`.  Every step of the
computation runs in the library's CUDA kernels; there is no other code path.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(HERE, "libssd.so")

SSD_F32, SSD_BF16 = 0, 1
STATUS = {0: "SSD_OK", 1: "SSD_ERR_NULL_ARG", 2: "SSD_ERR_INVALID_DIM", 3: "SSD_ERR_UNSUPPORTED",
          4: "SSD_ERR_MISALIGNED", 5: "SSD_ERR_CUDA", 6: "SSD_ERR_DEVICE_TIMEOUT",
          7: "SSD_ERR_WORKSPACE"}

EXPORTS = ("ssd_forward", "ssd_forward_ws", "ssd_forward_stage", "ssd_workspace_bytes",
           "ssd_workspace_layout", "ssd_device_status", "ssd_status_string", "ssd_version",
           "ssd_forward_static", "ssd_step", "ssd_forward_block", "ssd_block_workspace_bytes",
           "ssd_forward_varlen", "ssd_varlen_workspace_bytes", "ssd_backward", "ssd_workspace_trim",
           "ssd_glr_forward", "ssd_glr_backward", "ssd_glr_step", "ssd_glr_chunk_rows", "ssd_pack8", "ssd_unpack8",
           "ssd_norm_rotate", "ssd_norm_rotate_backward", "ssd_backward_packed8")
STAGES = ("ssd_chunk_cumsum", "ssd_chunk_state", "ssd_state_passing", "ssd_chunk_scan")


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_size_t), ("l_offset", ctypes.c_size_t),
                ("w_offset", ctypes.c_size_t), ("dtq_offset", ctypes.c_size_t),
                ("beta_offset", ctypes.c_size_t),
                ("alpha_offset", ctypes.c_size_t),
                ("states_offset", ctypes.c_size_t), ("s_in_offset", ctypes.c_size_t),
                ("s_in_dtype", ctypes.c_int32), ("tensor_core", ctypes.c_int32),
                ("launches", ctypes.c_int32), ("states_dtype", ctypes.c_int32),
                ("fused_state", ctypes.c_int32), ("single_pass", ctypes.c_int32),
                ("scan_engine", ctypes.c_int32), ("chunk_len", ctypes.c_int32)]


# ssd_scan_engine_t: which kernel computes y
SCAN_ENGINES = {0: "simt", 1: "tile", 2: "block_factored", 3: "chunk_wide", 4: "single_pass"}


class BlockOpts(ctypes.Structure):
    """ssd_block_opts_t: the scan's neighbours in the Mamba-2 block."""
    _fields_ = [("dt_bias", ctypes.c_void_p), ("dt_softplus", ctypes.c_int32),
                ("norm_apply", ctypes.c_int32), ("z", ctypes.c_void_p),
                ("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float),
                ("reserved0", ctypes.c_int32), ("rstd_out", ctypes.c_void_p)]


class GlrDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class RotateDims(ctypes.Structure):
    """ssd_rotate_dims_t: sizes and strides of a norm and rotation of B and C."""
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("rotary", ctypes.c_int64),
                ("B_batch_stride", ctypes.c_int64), ("B_token_stride", ctypes.c_int64),
                ("C_batch_stride", ctypes.c_int64), ("C_token_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class _Packed8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("exps", ctypes.c_void_p)]


class SSDError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libssd.so (raises if it has not been built; there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                           "`python -m structured_state_space_mamba_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, fp = ctypes.c_void_p, ctypes.c_void_p
    dims_p = ctypes.POINTER(Dims)
    lib.ssd_forward.argtypes = [dims_p, vp, fp, fp, vp, vp, fp, ctypes.c_int, fp, vp, fp, vp]
    lib.ssd_forward.restype = ctypes.c_int
    lib.ssd_forward_ws.argtypes = [dims_p, vp, fp, fp, vp, vp, fp, ctypes.c_int, fp, vp, fp,
                                   vp, ctypes.c_size_t, vp]
    lib.ssd_forward_ws.restype = ctypes.c_int
    lib.ssd_forward_static.argtypes = lib.ssd_forward.argtypes
    lib.ssd_forward_static.restype = ctypes.c_int
    lib.ssd_step.argtypes = [dims_p, vp, fp, fp, vp, vp, fp, fp, vp, vp]
    lib.ssd_step.restype = ctypes.c_int
    lib.ssd_forward_stage.argtypes = [ctypes.c_int] + lib.ssd_forward_ws.argtypes
    lib.ssd_forward_stage.restype = ctypes.c_int
    lib.ssd_forward_block.argtypes = [dims_p, vp, fp, fp, vp, vp, fp, ctypes.c_int, fp, vp, fp,
                                      ctypes.POINTER(BlockOpts), vp, ctypes.c_size_t, vp]
    lib.ssd_forward_block.restype = ctypes.c_int
    lib.ssd_block_workspace_bytes.argtypes = [dims_p, ctypes.c_int, ctypes.POINTER(BlockOpts)]
    lib.ssd_block_workspace_bytes.restype = ctypes.c_size_t
    i64p = ctypes.POINTER(ctypes.c_int64)
    lib.ssd_forward_varlen.argtypes = [dims_p, i64p, ctypes.c_int64, vp, fp, fp, vp, vp, fp, ctypes.c_int, fp,
                                       vp, fp, vp, ctypes.c_size_t, vp]
    lib.ssd_forward_varlen.restype = ctypes.c_int
    lib.ssd_varlen_workspace_bytes.argtypes = [dims_p, i64p, ctypes.c_int64, ctypes.c_int]
    lib.ssd_varlen_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_backward.argtypes = [dims_p, vp, fp, fp, vp, vp, fp, ctypes.c_int, fp, vp, fp, vp, fp, fp, vp, vp, fp,
                                 fp, vp]
    lib.ssd_backward.restype = ctypes.c_int
    lib.ssd_workspace_bytes.argtypes = [dims_p, ctypes.c_int]
    lib.ssd_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_workspace_layout.argtypes = [dims_p, ctypes.c_int, ctypes.POINTER(WorkspaceLayout)]
    lib.ssd_workspace_layout.restype = ctypes.c_int
    lib.ssd_status_string.argtypes = [ctypes.c_int]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_device_status.argtypes = [ctypes.c_void_p]
    lib.ssd_device_status.restype = ctypes.c_int
    lib.ssd_version.argtypes = []
    lib.ssd_version.restype = ctypes.c_char_p
    lib.ssd_workspace_trim.argtypes = []
    lib.ssd_workspace_trim.restype = ctypes.c_int
    i64, packed_p = ctypes.c_int64, ctypes.POINTER(_Packed8)
    glr_p, rot_p = ctypes.POINTER(GlrDims), ctypes.POINTER(RotateDims)
    lib.ssd_glr_forward.argtypes = [glr_p, vp, i64, vp, vp, vp, fp, fp, vp, fp, fp, packed_p, vp]
    lib.ssd_glr_backward.argtypes = [glr_p, vp, i64, vp, vp, vp, packed_p, fp, fp, vp, fp, vp, vp, vp, fp, fp, vp]
    lib.ssd_glr_step.argtypes = [glr_p, vp, vp, vp, fp, fp, vp, vp]
    lib.ssd_glr_chunk_rows.argtypes = [glr_p, vp, i64]
    lib.ssd_glr_chunk_rows.restype = i64
    lib.ssd_pack8.argtypes = [i64, i64, ctypes.c_int, vp, packed_p, vp]
    lib.ssd_unpack8.argtypes = [i64, i64, ctypes.c_int, packed_p, vp, vp]
    lib.ssd_norm_rotate.argtypes = [rot_p, vp, vp, vp, fp, fp, fp, vp, vp, vp]
    lib.ssd_norm_rotate_backward.argtypes = [rot_p, vp, vp, vp, vp, vp, fp, fp, fp, vp, vp, fp, fp, vp]
    lib.ssd_backward_packed8.argtypes = [dims_p, packed_p, fp, fp, fp, ctypes.c_int, fp, vp, fp, vp, fp, fp, vp, vp,
                                         fp, fp, vp]
    for f in (lib.ssd_backward_packed8, lib.ssd_glr_forward, lib.ssd_glr_backward, lib.ssd_glr_step, lib.ssd_pack8, lib.ssd_unpack8,
              lib.ssd_norm_rotate, lib.ssd_norm_rotate_backward):
        f.restype = ctypes.c_int
    _lib = lib
    return lib


def make_dims(batch, seqlen, nheads, headdim, dstate, ngroups, dtype) -> Dims:
    code = {"f32": SSD_F32, "bf16": SSD_BF16, torch.float32: SSD_F32,
            torch.bfloat16: SSD_BF16}[dtype]
    return Dims(batch, seqlen, nheads, headdim, dstate, ngroups, code, 0)


def _check(status: int):
    if status != 0:
        raise SSDError(status, load().ssd_status_string(status).decode())


def workspace_bytes(dims: Dims, chunk_len: int) -> int:
    return int(load().ssd_workspace_bytes(ctypes.byref(dims), int(chunk_len)))


def workspace_layout(dims: Dims, chunk_len: int) -> WorkspaceLayout:
    out = WorkspaceLayout()
    _check(load().ssd_workspace_layout(ctypes.byref(dims), int(chunk_len), ctypes.byref(out)))
    return out


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _validate(x, dt, A, B, C, D, init_state):
    if not x.is_cuda:
        raise ValueError("ssd.forward runs on CUDA tensors only")
    dev = x.device
    for name, t in (("dt", dt), ("A", A), ("B", B), ("C", C), ("D", D),
                    ("init_state", init_state)):
        if t is None:
            continue
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, x on {dev}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if x.dtype not in (torch.float32, torch.bfloat16) or B.dtype != x.dtype or C.dtype != x.dtype:
        raise ValueError("x, B and C must share a dtype: float32 or bfloat16")
    for name, t in (("dt", dt), ("A", A), ("D", D), ("init_state", init_state)):
        if t is not None and t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32")
    bsz, T, H, P = x.shape
    if B.dim() != 4 or B.shape[:2] != (bsz, T) or C.shape != B.shape:
        raise ValueError("B and C must be [batch, seqlen, ngroups, dstate]")
    G, N = B.shape[2], B.shape[3]
    if dt.shape != (bsz, T, H) or A.shape != (H,):
        raise ValueError("dt must be [batch, seqlen, nheads] and A [nheads]")
    if D is not None and D.shape != (H,):
        raise ValueError("D must be [nheads]")
    if init_state is not None and init_state.shape != (bsz, H, P, N):
        raise ValueError("init_state must be [batch, nheads, headdim, dstate]")
    return make_dims(bsz, T, H, P, N, G, x.dtype)


def forward(x, dt, A, B, C, D=None, chunk_len=256, init_state=None, return_final_state=False,
            out=None, final_out=None, workspace=None, stream=None, stage=None):
    """y (and optionally the final state) of the SSD forward scan.

    x [B,T,H,P], B/C [B,T,G,N] (float32 or bfloat16); dt [B,T,H], A [H], D [H],
    init_state [B,H,P,N] float32.  Returns ``y`` or ``(y, final_state)``.
    ``workspace``: optional uint8 CUDA tensor of at least ``workspace_bytes``
    bytes (otherwise the library allocates it stream-ordered).
    """
    dims = _validate(x, dt, A, B, C, D, init_state)
    y = out if out is not None else torch.empty_like(x)
    fin = final_out
    if fin is None and return_final_state:
        fin = torch.empty((dims.batch, dims.nheads, dims.headdim, dims.dstate),
                          dtype=torch.float32, device=x.device)
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    lib = load()
    args = [ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
            int(chunk_len), _ptr(init_state), _ptr(y), _ptr(fin)]
    with torch.cuda.device(x.device):
        if stage is not None:
            if workspace is None:
                raise ValueError("a single stage needs workspace=")
            st = lib.ssd_forward_stage(int(stage), *args, _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       ctypes.c_void_p(stream))
        elif workspace is None:
            st = lib.ssd_forward(*args, ctypes.c_void_p(stream))
        else:
            st = lib.ssd_forward_ws(*args, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    ctypes.c_void_p(stream))
    _check(st)
    if return_final_state or final_out is not None:
        return y, fin
    return y


def forward_block(x, dt, A, B, C, D=None, chunk_len=256, init_state=None, dt_bias=None,
                  dt_softplus=False, z=None, norm_weight=None, norm_eps=1e-5, norm_apply=True,
                  return_rstd=False, return_final_state=False, out=None, final_out=None,
                  workspace=None, stream=None):
    """The scan with its block neighbours through ``ssd_forward_block``:
    softplus(dt + dt_bias) as the step size, then y * silu(z) and RMSNorm over
    each token's H * P values with ``norm_weight`` [H*P] float32.  With
    ``norm_apply=False`` the output is the gated, weighted y and the per-token
    factor rstd [B, T] is returned for the caller to apply.
    Returns ``out`` plus, as asked, the final state and rstd (in that order)."""
    dims = _validate(x, dt, A, B, C, D, init_state)
    dev = x.device
    for name, t in (("dt_bias", dt_bias), ("norm_weight", norm_weight)):
        if t is not None and (t.device != dev or t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor on {dev}")
    if z is not None and (z.device != dev or z.dtype != x.dtype or z.shape != x.shape or not z.is_contiguous()):
        raise ValueError("z must be a contiguous tensor like x")
    y = out if out is not None else torch.empty_like(x)
    fin = final_out
    if fin is None and return_final_state:
        fin = torch.empty((dims.batch, dims.nheads, dims.headdim, dims.dstate),
                          dtype=torch.float32, device=dev)
    rstd = None
    if norm_weight is not None and (return_rstd or not norm_apply):
        rstd = torch.empty((dims.batch, dims.seqlen), dtype=torch.float32, device=dev)
    opts = BlockOpts(dt_bias=None if dt_bias is None else dt_bias.data_ptr(),
                     dt_softplus=1 if dt_softplus else 0, norm_apply=1 if norm_apply else 0,
                     z=None if z is None else z.data_ptr(),
                     norm_weight=None if norm_weight is None else norm_weight.data_ptr(),
                     norm_eps=float(norm_eps), reserved0=0,
                     rstd_out=None if rstd is None else rstd.data_ptr())
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    with torch.cuda.device(dev):
        wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
        st = load().ssd_forward_block(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                      _ptr(D), int(chunk_len), _ptr(init_state), _ptr(y), _ptr(fin),
                                      ctypes.byref(opts), _ptr(workspace), wsz, ctypes.c_void_p(stream))
    _check(st)
    res = [y]
    if return_final_state or final_out is not None:
        res.append(fin)
    if rstd is not None:
        res.append(rstd)
    return res[0] if len(res) == 1 else tuple(res)


def _cu_array(cu_seqlens):
    import numpy as np
    cu = np.ascontiguousarray(np.asarray(cu_seqlens.cpu() if isinstance(cu_seqlens, torch.Tensor) else cu_seqlens,
                                         dtype=np.int64))
    if cu.ndim != 1 or cu.size < 2:
        raise ValueError("cu_seqlens must be a 1-D array of nseq + 1 offsets")
    return cu


def varlen_workspace_bytes(dims: Dims, cu_seqlens, chunk_len: int) -> int:
    cu = _cu_array(cu_seqlens)
    return int(load().ssd_varlen_workspace_bytes(ctypes.byref(dims), cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                                 cu.size - 1, int(chunk_len)))


def forward_varlen(x, dt, A, B, C, cu_seqlens, D=None, chunk_len=256, init_states=None,
                   return_final_states=False, out=None, final_out=None, workspace=None, stream=None):
    """Several sequences packed along the token axis through ``ssd_forward_varlen``.

    x [1, T, H, P], dt [1, T, H], B/C [1, T, G, N]; ``cu_seqlens`` (host: a list,
    a numpy array or a CPU tensor) holds nseq + 1 offsets; ``init_states`` and
    the final states are [nseq, H, P, N] float32.  Returns y (and the final
    states)."""
    cu = _cu_array(cu_seqlens)
    nseq = cu.size - 1
    dims = _validate(x, dt, A, B, C, D, None)
    dev = x.device
    st_shape = (nseq, dims.nheads, dims.headdim, dims.dstate)
    if init_states is not None and (init_states.device != dev or init_states.dtype != torch.float32
                                    or tuple(init_states.shape) != st_shape or not init_states.is_contiguous()):
        raise ValueError(f"init_states must be a contiguous float32 tensor {st_shape} on {dev}")
    y = out if out is not None else torch.empty_like(x)
    fin = final_out
    if fin is None and return_final_states:
        fin = torch.empty(st_shape, dtype=torch.float32, device=dev)
    cu_p = cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))
    if workspace is None:
        need = int(load().ssd_varlen_workspace_bytes(ctypes.byref(dims), cu_p, nseq, int(chunk_len)))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    with torch.cuda.device(dev):
        wsz = workspace.numel() * workspace.element_size()
        st = load().ssd_forward_varlen(ctypes.byref(dims), cu_p, nseq, _ptr(x), _ptr(dt), _ptr(A), _ptr(B),
                                       _ptr(C), _ptr(D), int(chunk_len), _ptr(init_states), _ptr(y), _ptr(fin),
                                       _ptr(workspace), wsz, ctypes.c_void_p(stream))
    _check(st)
    return (y, fin) if (return_final_states or final_out is not None) else y


def backward(x, dt, A, B, C, dy, D=None, chunk_len=256, init_state=None, dfinal_state=None, stream=None):
    """Gradients through ``ssd_backward``: returns a dict with dx, ddt, dA, dB,
    dC, dD (None without D) and dinit_state (None without an initial state)."""
    dims = _validate(x, dt, A, B, C, D, init_state)
    dev = x.device
    if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != dev or not dy.is_contiguous():
        raise ValueError("dy must be a contiguous tensor like x")
    if dfinal_state is not None and (dfinal_state.dtype != torch.float32 or not dfinal_state.is_contiguous()
                                     or tuple(dfinal_state.shape) != (dims.batch, dims.nheads, dims.headdim,
                                                                      dims.dstate)):
        raise ValueError("dfinal_state must be a contiguous float32 [batch, nheads, headdim, dstate] tensor")
    out = dict(dx=torch.empty_like(x), ddt=torch.empty_like(dt), dA=torch.empty_like(A),
               dB=torch.empty_like(B), dC=torch.empty_like(C),
               dD=None if D is None else torch.empty_like(D),
               dinit_state=None if init_state is None else torch.empty_like(init_state))
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    with torch.cuda.device(dev):
        st = load().ssd_backward(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                 int(chunk_len), _ptr(init_state), _ptr(dy), _ptr(dfinal_state), _ptr(out["dx"]),
                                 _ptr(out["ddt"]), _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]),
                                 _ptr(out["dD"]), _ptr(out["dinit_state"]), ctypes.c_void_p(stream))
    _check(st)
    return out


def block_workspace_bytes(dims: Dims, chunk_len: int, dt_transform: bool) -> int:
    opts = BlockOpts(dt_softplus=1 if dt_transform else 0)
    return int(load().ssd_block_workspace_bytes(ctypes.byref(dims), int(chunk_len), ctypes.byref(opts)))


def forward_ws(*args, **kwargs):
    """``forward`` with a required ``workspace`` keyword."""
    if kwargs.get("workspace") is None:
        raise ValueError("forward_ws needs workspace=")
    return forward(*args, **kwargs)


def forward_static(x, dt, A, B, C, D=None, chunk_len=256, init_state=None,
                   return_final_state=False, out=None, final_out=None, stream=None):
    """``forward`` through ``ssd_forward_static``: the intermediates live in the
    library's fixed per-device scratch array, and nothing is allocated.  A
    workload whose workspace exceeds ``STATIC_SCRATCH_BYTES`` raises (status
    SSD_ERR_WORKSPACE); calls that overlap in time on one device race on the
    shared scratch."""
    dims = _validate(x, dt, A, B, C, D, init_state)
    y = out if out is not None else torch.empty_like(x)
    fin = final_out
    if fin is None and return_final_state:
        fin = torch.empty((dims.batch, dims.nheads, dims.headdim, dims.dstate),
                          dtype=torch.float32, device=x.device)
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    with torch.cuda.device(x.device):
        st = load().ssd_forward_static(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B),
                                       _ptr(C), _ptr(D), int(chunk_len), _ptr(init_state),
                                       _ptr(y), _ptr(fin), ctypes.c_void_p(stream))
    _check(st)
    if return_final_state or final_out is not None:
        return y, fin
    return y


STATIC_SCRATCH_BYTES = 64 << 20  # SSD_STATIC_SCRATCH_BYTES in include/ssd.h


def step(state, x, dt, A, B, C, D=None, out=None, stream=None):
    """One decode step through ``ssd_step``: ``state`` [B,H,P,N] float32 is
    updated in place to exp(dt A) state + dt x B^T and y = state C + D x is
    returned.  x [B,H,P], B/C [B,G,N] (float32 or bfloat16, one dtype);
    dt [B,H], A [H], D [H] float32."""
    if not x.is_cuda:
        raise ValueError("ssd.step runs on CUDA tensors only")
    dev = x.device
    for name, t in (("state", state), ("dt", dt), ("A", A), ("B", B), ("C", C), ("D", D)):
        if t is None:
            continue
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, x on {dev}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if x.dtype not in (torch.float32, torch.bfloat16) or B.dtype != x.dtype or C.dtype != x.dtype:
        raise ValueError("x, B and C must share a dtype: float32 or bfloat16")
    for name, t in (("state", state), ("dt", dt), ("A", A), ("D", D)):
        if t is not None and t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32")
    bsz, H, P = x.shape
    if B.dim() != 3 or B.shape[0] != bsz or C.shape != B.shape:
        raise ValueError("B and C must be [batch, ngroups, dstate]")
    G, N = B.shape[1], B.shape[2]
    if dt.shape != (bsz, H) or A.shape != (H,) or state.shape != (bsz, H, P, N):
        raise ValueError("dt must be [batch, nheads], A [nheads], state [batch, nheads, headdim, dstate]")
    if D is not None and D.shape != (H,):
        raise ValueError("D must be [nheads]")
    dims = make_dims(bsz, 1, H, P, N, G, x.dtype)
    y = out if out is not None else torch.empty_like(x)
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    with torch.cuda.device(dev):
        st = load().ssd_step(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                             _ptr(state), _ptr(y), ctypes.c_void_p(stream))
    _check(st)
    return y


# ---------------------------------------------------------------------------
# gated linear recurrence, 8-bit checkpoints, norm and rotation of B and C
# ---------------------------------------------------------------------------
GLR_CHUNK = 64    # SSD_GLR_CHUNK in include/ssd.h
PACK8_BLOCK = 64  # SSD_PACK8_BLOCK in include/ssd.h
_CODE = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}


_get_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _is(t, index, dtype, shape):
    """Whether t is a contiguous tensor of that dtype and shape on that CUDA device."""
    return t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _need(name, t, index, dtype, shape):
    """Refuses a tensor for which ``_is`` does not hold, with what is wrong."""
    if _is(t, index, dtype, shape):
        return
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, is {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, is {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _storage(name, x):
    """(ssd_dtype_t, CUDA device index) of a tensor in a storage type."""
    index, code = x.get_device(), _CODE.get(x.dtype)
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return code, index


def _ptr_or_none(t):
    return None if t is None else t.data_ptr()


def _launch(index, stream, call, *args):
    """call(stream, *args) with the tensors' device current.  With a stream other
    than the current one (a torch stream, or its handle) the outputs are
    allocated for it, so that memory which the current stream still uses is not
    taken."""
    if _get_device() != index:
        with torch.cuda.device(index):
            return _launch(index, stream, call, *args)
    current = _raw_stream(index)
    if stream is not None:
        handle = int(getattr(stream, "cuda_stream", stream))
        if handle != current:
            other = torch.cuda.ExternalStream(handle, device=index) if handle else torch.cuda.default_stream(index)
            with torch.cuda.stream(other):
                return call(handle, *args)
    return call(current, *args)


class Packed8:
    """An activation [..., channels] in 8 bits (``pack8``): ``codes`` int8 of its
    shape and ``exps`` uint8 [..., ceil(channels / 64)], one power-of-two step a
    block of 64 values."""
    __slots__ = ("codes", "exps")

    def __init__(self, codes, exps):
        self.codes, self.exps = codes, exps

    @classmethod
    def empty_like(cls, x):
        return cls(x.new_empty(x.shape, dtype=torch.int8),
                   x.new_empty((*x.shape[:-1], -(-x.shape[-1] // PACK8_BLOCK)), dtype=torch.uint8))

    @property
    def shape(self):
        return self.codes.shape

    def _c(self):
        return _Packed8(self.codes.data_ptr(), self.exps.data_ptr())

    def _check(self, name, index, shape):
        _need(f"{name}.codes", self.codes, index, torch.int8, shape)
        _need(f"{name}.exps", self.exps, index, torch.uint8, (*shape[:-1], -(-shape[-1] // PACK8_BLOCK)))


def pack8(x, stream=None):
    """``x`` [..., channels] (float32 or bfloat16) as an 8-bit checkpoint: one
    signed byte a value and one power-of-two step for every 64 values of a row,
    off by at most 1/127.5 of the largest magnitude among them."""
    code, index = _storage("x", x)
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be contiguous with at least one dimension")
    return _launch(index, stream, _pack8, x, code)


def _pack8(st, x, code):
    cols = x.shape[-1]
    p = Packed8.empty_like(x)
    _check(load().ssd_pack8(x.numel() // cols if cols else 0, cols, code, x.data_ptr(), ctypes.byref(p._c()), st))
    return p


def unpack8(packed, dtype=torch.bfloat16, out=None, stream=None):
    """The values of a checkpoint in float32 or bfloat16 (exact in either)."""
    if not isinstance(packed, Packed8):
        raise ValueError("packed must be a Packed8")
    index = packed.codes.get_device()
    if index < 0 or packed.codes.dim() < 1:
        raise ValueError("packed must hold CUDA tensors of at least one dimension")
    packed._check("packed", index, packed.shape)
    if dtype not in _CODE:
        raise ValueError("dtype must be float32 or bfloat16")
    if out is not None:
        _need("out", out, index, dtype, packed.shape)
    return _launch(index, stream, _unpack8, packed, dtype, out)


def _unpack8(st, packed, dtype, out):
    cols = packed.shape[-1]
    if out is None:
        out = packed.codes.new_empty(packed.shape, dtype=dtype)
    _check(load().ssd_unpack8(packed.codes.numel() // cols if cols else 0, cols, _CODE[dtype],
                              ctypes.byref(packed._c()), out.data_ptr(), st))
    return out


def backward_packed8(x, dt, A, B, C, dy, D=None, chunk_len=256, init_state=None, dfinal_state=None, stream=None):
    """``backward`` from 8-bit checkpoints (``pack8``) of x, B and C through
    ``ssd_backward_packed8``: the gradients at the values that they stand for,
    in dy's dtype.  Reads them back into scratch first.  Returns the dict of
    ``backward``."""
    code, index = _storage("dy", dy)
    if dy.dim() != 4:
        raise ValueError("dy must be [batch, seqlen, nheads, headdim]")
    for name, p in (("x", x), ("B", B), ("C", C)):
        if not isinstance(p, Packed8):
            raise ValueError(f"{name} must be a Packed8")
    bsz, T, H, P = dy.shape
    if B.codes.dim() != 4:
        raise ValueError("B and C must be [batch, seqlen, ngroups, dstate]")
    G, N = B.shape[2:]
    _need("dy", dy, index, dy.dtype, dy.shape)
    x._check("x", index, dy.shape)
    B._check("B", index, (bsz, T, G, N))
    C._check("C", index, (bsz, T, G, N))
    for name, t, shape in (("dt", dt, (bsz, T, H)), ("A", A, (H,)), ("D", D, (H,)),
                           ("init_state", init_state, (bsz, H, P, N)),
                           ("dfinal_state", dfinal_state, (bsz, H, P, N))):
        if t is not None:
            _need(name, t, index, torch.float32, shape)
    return _launch(index, stream, _backward_packed8, Dims(bsz, T, H, P, N, G, code, 0), x, dt, A, B, C, dy, D,
                   int(chunk_len), init_state, dfinal_state)


def _backward_packed8(st, dims, x, dt, A, B, C, dy, D, chunk_len, init_state, dfinal_state):
    out = dict(dx=torch.empty_like(dy), ddt=torch.empty_like(dt), dA=torch.empty_like(A),
               dB=dy.new_empty(B.shape), dC=dy.new_empty(C.shape), dD=None if D is None else torch.empty_like(D),
               dinit_state=None if init_state is None else torch.empty_like(init_state))
    pk = (_Packed8 * 3)(x._c(), B._c(), C._c())
    _check(load().ssd_backward_packed8(
        ctypes.byref(dims), pk, dt.data_ptr(), A.data_ptr(), _ptr_or_none(D), chunk_len, _ptr_or_none(init_state),
        dy.data_ptr(), _ptr_or_none(dfinal_state), out["dx"].data_ptr(), out["ddt"].data_ptr(), out["dA"].data_ptr(),
        out["dB"].data_ptr(), out["dC"].data_ptr(), _ptr_or_none(out["dD"]), _ptr_or_none(out["dinit_state"]), st))
    return out


class GlrSaved:
    """What ``glr_forward`` keeps for ``glr_backward``: the inputs, or their 8-bit
    checkpoints, and the state entering every 64 tokens of every sequence."""
    __slots__ = ("x", "r", "i", "A", "chunk_states", "cu", "rows")

    def __init__(self, x, r, i, A, chunk_states, cu, rows):
        self.x, self.r, self.i, self.A, self.chunk_states, self.cu, self.rows = x, r, i, A, chunk_states, cu, rows


def glr_forward(x, r, i, A, init_state=None, cu_seqlens=None, return_final_state=False, save=None, out=None,
                stream=None):
    """The gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(i_t) x_t with
    a_t = exp(A s(r_t)), s the logistic function, through ``ssd_glr_forward``.

    x, r, i [B, T, C] (float32 or bfloat16, one dtype; contiguous, on 16 bytes);
    A [C] float32, at most 0; ``cu_seqlens`` (host: a list, a numpy array or a CPU tensor; B must be 1)
    holds nseq + 1 offsets of sequences packed along T; init_state and the final
    state are [B or nseq, C] float32.  ``save`` keeps what ``glr_backward`` needs:
    "inputs" refers to x, r and i themselves, "packed8" writes 8-bit
    checkpoints of them in the same pass.  Returns y plus, as asked, the final
    state and the saved (in that order)."""
    code, index = _storage("x", x)
    shape, dtype = x.shape, x.dtype
    if len(shape) != 3:
        raise ValueError("x must be [batch, seqlen, channels]")
    for name, t in (("x", x), ("r", r), ("i", i)):
        _need(name, t, index, dtype, shape)
    B, T, C = shape
    _need("A", A, index, torch.float32, (C,))
    if save not in (None, "inputs", "packed8"):
        raise ValueError('save must be None, "inputs" or "packed8"')
    cu = None if cu_seqlens is None else _cu_array(cu_seqlens)
    rows = B if cu is None else cu.size - 1
    if init_state is not None:
        _need("init_state", init_state, index, torch.float32, (rows, C))
    if out is not None:
        _need("out", out, index, dtype, shape)
    return _launch(index, stream, _glr_forward, GlrDims(B, T, C, code, 0), x, r, i, A, init_state, cu, rows,
                   return_final_state, save, out)


def _glr_forward(st, dims, x, r, i, A, init_state, cu, rows, return_final_state, save, out):
    lib, C = load(), dims.channels
    cu_p, nseq = (None, 0) if cu is None else (cu.ctypes.data, rows)
    y = torch.empty_like(x) if out is None else out
    final = A.new_empty(rows, C) if return_final_state else None
    states = packed = pk = None
    if save is not None:
        states = A.new_empty(lib.ssd_glr_chunk_rows(ctypes.byref(dims), cu_p, nseq), C)
        if save == "packed8":
            packed = [Packed8.empty_like(x) for _ in range(3)]
            pk = (_Packed8 * 3)(*(p._c() for p in packed))
    _check(lib.ssd_glr_forward(ctypes.byref(dims), cu_p, nseq, x.data_ptr(), r.data_ptr(), i.data_ptr(),
                               A.data_ptr(), _ptr_or_none(init_state), y.data_ptr(), _ptr_or_none(final),
                               _ptr_or_none(states), pk, st))
    if save is None:
        return (y, final) if return_final_state else y
    # the offsets are kept too: a copy, as they may be the caller's own array
    saved = GlrSaved(*(packed or (x, r, i)), A, states, None if cu is None else cu.copy(), rows)
    return (y, final, saved) if return_final_state else (y, saved)


def glr_backward(dy, saved, dfinal_state=None, return_dinit_state=False, stream=None):
    """Gradients of ``glr_forward`` through ``ssd_glr_backward``, from what it saved
    and the cotangents dy [B, T, C] and dfinal_state [B or nseq, C]: a dict with
    dx, dr, di (dy's dtype), dA, and dinit_state (None unless asked for)."""
    if not isinstance(saved, GlrSaved):
        raise ValueError("saved must be what glr_forward returned with save=")
    code, index = _storage("dy", dy)
    shape, dtype = dy.shape, dy.dtype
    if len(shape) != 3:
        raise ValueError("dy must be [batch, seqlen, channels]")
    _need("dy", dy, index, dtype, shape)
    B, T, C = shape
    packed = isinstance(saved.x, Packed8)
    for name, t in (("the saved x", saved.x), ("the saved r", saved.r), ("the saved i", saved.i)):
        if packed:
            t._check(name, index, shape)
        else:
            _need(name, t, index, dtype, shape)
    _need("the saved A", saved.A, index, torch.float32, (C,))
    if dfinal_state is not None:
        _need("dfinal_state", dfinal_state, index, torch.float32, (saved.rows, C))
    return _launch(index, stream, _glr_backward, GlrDims(B, T, C, code, 0), dy, saved, packed, dfinal_state,
                   return_dinit_state, index)


def _glr_backward(st, dims, dy, saved, packed, dfinal_state, return_dinit_state, index):
    lib, C, cu = load(), dims.channels, saved.cu
    cu_p, nseq = (None, 0) if cu is None else (cu.ctypes.data, saved.rows)
    _need("the saved chunk_states", saved.chunk_states, index, torch.float32,
          (lib.ssd_glr_chunk_rows(ctypes.byref(dims), cu_p, nseq), C))
    dx, dr, di = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(dy)
    dA = torch.empty_like(saved.A)
    dinit = saved.A.new_empty(saved.rows, C) if return_dinit_state else None
    if packed:
        x = r = i = None
        pk = (_Packed8 * 3)(saved.x._c(), saved.r._c(), saved.i._c())
    else:
        x, r, i, pk = saved.x.data_ptr(), saved.r.data_ptr(), saved.i.data_ptr(), None
    _check(lib.ssd_glr_backward(ctypes.byref(dims), cu_p, nseq, x, r, i, pk, saved.A.data_ptr(),
                                saved.chunk_states.data_ptr(), dy.data_ptr(), _ptr_or_none(dfinal_state),
                                dx.data_ptr(), dr.data_ptr(), di.data_ptr(), dA.data_ptr(), _ptr_or_none(dinit), st))
    return dict(dx=dx, dr=dr, di=di, dA=dA, dinit_state=dinit)


def glr_step(state, x, r, i, A, out=None, stream=None):
    """One token of the gated linear recurrence through ``ssd_glr_step``: ``state``
    [B, C] float32 is updated in place and the output is returned.  x, r, i
    [B, C] (float32 or bfloat16, one dtype; contiguous, on 16 bytes); A [C] float32."""
    code, index = _storage("x", x)
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2:
        raise ValueError("x must be [batch, channels]")
    for name, t in (("x", x), ("r", r), ("i", i)):
        _need(name, t, index, dtype, shape)
    _need("A", A, index, torch.float32, shape[1:])
    _need("state", state, index, torch.float32, shape)
    if out is not None:
        _need("out", out, index, dtype, shape)
    return _launch(index, stream, _glr_step, GlrDims(shape[0], 1, shape[1], code, 0), state, x, r, i, A, out)


def _glr_step(st, dims, state, x, r, i, A, out):
    y = torch.empty_like(x) if out is None else out
    _check(load().ssd_glr_step(ctypes.byref(dims), x.data_ptr(), r.data_ptr(), i.data_ptr(), A.data_ptr(),
                               state.data_ptr(), y.data_ptr(), st))
    return y


def _rotate_dims(B, C, positions, inv_freq, weight_B, weight_C, eps, interleaved):
    code, index = _storage("B", B)
    shape = B.shape
    if len(shape) != 4:
        raise ValueError("B and C must be [batch, seqlen, ngroups, dstate]")
    if C.get_device() != index or C.dtype is not B.dtype or C.shape != shape:
        raise ValueError("B and C must have one shape, dtype and device")
    bsz, T, G, N = shape
    b0, b1, b2, b3 = B.stride()
    c0, c1, c2, c3 = C.stride()
    if (N > 1 and (b3 != 1 or c3 != 1)) or (G > 1 and (b2 != N or c2 != N)):
        raise ValueError("a token's values of B and of C must be contiguous")
    _need("positions", positions, index, torch.int64, (bsz, T))
    half = inv_freq.numel()
    _need("inv_freq", inv_freq, index, torch.float32, (half,))
    if weight_B is not None:
        _need("weight_B", weight_B, index, torch.float32, (N,))
    if weight_C is not None:
        _need("weight_C", weight_C, index, torch.float32, (N,))
    return index, RotateDims(bsz, T, G, N, 2 * half, b0, b1, c0, c1, code, 1 if interleaved else 0, eps, 0)


def norm_rotate(B, C, positions, inv_freq, weight_B=None, weight_C=None, eps=1e-5, interleaved=False, stream=None):
    """RMSNorm over dstate of every group's B and C and the position rotation,
    through ``ssd_norm_rotate``: what the scan takes as its B and C.

    B, C [batch, seqlen, ngroups, dstate] (float32 or bfloat16; slices of a
    projection's rows are taken as they are); positions [batch, seqlen] int64;
    inv_freq [rotary / 2] float32, rotary at most dstate; weights [dstate]
    float32 or None.  Pairs are (j, j + rotary / 2), or neighbours with
    ``interleaved``.  Returns (B, C), contiguous."""
    index, dims = _rotate_dims(B, C, positions, inv_freq, weight_B, weight_C, eps, interleaved)
    return _launch(index, stream, _norm_rotate, dims, B, C, positions, inv_freq, weight_B, weight_C)


def _norm_rotate(st, dims, B, C, positions, inv_freq, weight_B, weight_C):
    Bo, Co = (torch.empty_like(t, memory_format=torch.contiguous_format) for t in (B, C))
    _check(load().ssd_norm_rotate(ctypes.byref(dims), B.data_ptr(), C.data_ptr(), positions.data_ptr(),
                                  inv_freq.data_ptr() or None, _ptr_or_none(weight_B), _ptr_or_none(weight_C),
                                  Bo.data_ptr(), Co.data_ptr(), st))
    return Bo, Co


def norm_rotate_backward(dB_out, dC_out, B, C, positions, inv_freq, weight_B=None, weight_C=None, eps=1e-5,
                         interleaved=False, stream=None):
    """Gradients of ``norm_rotate`` through ``ssd_norm_rotate_backward``, from the
    cotangents of its outputs and its inputs: a dict with dB, dC (contiguous),
    dweight_B and dweight_C (None without that weight)."""
    index, dims = _rotate_dims(B, C, positions, inv_freq, weight_B, weight_C, eps, interleaved)
    _need("dB_out", dB_out, index, B.dtype, B.shape)
    _need("dC_out", dC_out, index, B.dtype, B.shape)
    return _launch(index, stream, _norm_rotate_backward, dims, dB_out, dC_out, B, C, positions, inv_freq, weight_B,
                   weight_C)


def _norm_rotate_backward(st, dims, dB_out, dC_out, B, C, positions, inv_freq, weight_B, weight_C):
    dB, dC = torch.empty_like(dB_out), torch.empty_like(dC_out)
    dwB = None if weight_B is None else torch.empty_like(weight_B)
    dwC = None if weight_C is None else torch.empty_like(weight_C)
    _check(load().ssd_norm_rotate_backward(
        ctypes.byref(dims), dB_out.data_ptr(), dC_out.data_ptr(), B.data_ptr(), C.data_ptr(), positions.data_ptr(),
        inv_freq.data_ptr() or None, _ptr_or_none(weight_B), _ptr_or_none(weight_C), dB.data_ptr(), dC.data_ptr(),
        _ptr_or_none(dwB), _ptr_or_none(dwC), st))
    return dict(dB=dB, dC=dC, dweight_B=dwB, dweight_C=dwC)


def device_status(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device error
    status: 0 (SSD_OK) or 6 (SSD_ERR_DEVICE_TIMEOUT)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        return int(load().ssd_device_status(
            ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)))


def workspace_trim(device=None) -> int:
    """Synchronise the device and return the library pool's unused workspace
    memory to the system; 0 (SSD_OK) or an ssd_status_t error code."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        return int(load().ssd_workspace_trim())


def version() -> str:
    return load().ssd_version().decode()
