"""The C boundary of the gated linear recurrence, the 8-bit checkpoints and the
norm and rotation, on the CPU: every call here is refused by the host checks
before anything is launched, so the made-up addresses are never dereferenced.
"""
import ctypes

import numpy as np
import pytest
import torch

from structured_state_space_mamba_b200 import binding

NULL, INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3, 4
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from structured_state_space_mamba_b200 import build
    build.build()
    return binding.load()


def glr_dims(batch=2, seqlen=100, channels=65, dtype=1, reserved=0):
    return binding.GlrDims(batch, seqlen, channels, dtype, reserved)


def cu_array(cu):
    return None if cu is None else np.asarray(cu, dtype=np.int64)


def packed(codes=FAKE, exps=FAKE, last=FAKE):
    return (binding._Packed8 * 3)(binding._Packed8(codes, exps), binding._Packed8(FAKE, FAKE),
                                  binding._Packed8(FAKE, last))


def forward(lib, dims, cu=None, nseq=None, pk=None, **kw):
    p = dict(x=FAKE, r=FAKE, i=FAKE, A=FAKE, h0=None, y=FAKE, fin=None, st=None)
    p.update(kw)
    a = cu_array(cu)
    return lib.ssd_glr_forward(ctypes.byref(dims) if dims is not None else None,
                               None if a is None else a.ctypes.data, (len(a) - 1 if nseq is None else nseq) if a is not None else 0,
                               p["x"], p["r"], p["i"], p["A"], p["h0"], p["y"], p["fin"], p["st"], pk, None)


def backward(lib, dims, cu=None, pk=None, **kw):
    p = dict(x=FAKE, r=FAKE, i=FAKE, A=FAKE, st=FAKE, dy=FAKE, df=None, dx=FAKE, dr=FAKE, di=FAKE, dA=FAKE, dh=None)
    p.update(kw)
    a = cu_array(cu)
    return lib.ssd_glr_backward(ctypes.byref(dims), None if a is None else a.ctypes.data,
                                0 if a is None else len(a) - 1, p["x"], p["r"], p["i"], pk, p["A"], p["st"], p["dy"],
                                p["df"], p["dx"], p["dr"], p["di"], p["dA"], p["dh"], None)


BAD_GLR = [(dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(channels=-1), INVALID),
           (dict(reserved=1), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(seqlen=(1 << 30) + 1), UNSUPPORTED),
           (dict(channels=(1 << 24) + 1), UNSUPPORTED), (dict(batch=1 << 20, seqlen=1 << 20), UNSUPPORTED),
           (dict(batch=1 << 40), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_GLR, ids=str)
def test_glr_sizes(lib, kw, code):
    d = glr_dims(**kw)
    assert forward(lib, d) == code and backward(lib, d) == code
    assert lib.ssd_glr_chunk_rows(ctypes.byref(d), None, 0) == 0


@pytest.mark.parametrize("cu,batch", [([1, 100], 1), ([0, 99], 1), ([0, 60, 50, 100], 1), ([0, 101, 100], 1),
                                      ([0, 100], 2), ([0, -1, 100], 1)])
def test_glr_offsets(lib, cu, batch):
    d = glr_dims(batch=batch)
    assert forward(lib, d, cu) == INVALID and backward(lib, d, cu) == INVALID
    assert lib.ssd_glr_chunk_rows(ctypes.byref(d), cu_array(cu).ctypes.data, len(cu) - 1) == 0


def test_glr_no_sequences(lib):
    assert forward(lib, glr_dims(batch=1), [0, 100], nseq=0) == INVALID
    assert forward(lib, None) == NULL


def test_glr_chunk_rows(lib):
    d = glr_dims(batch=3, seqlen=129)
    assert lib.ssd_glr_chunk_rows(ctypes.byref(d), None, 0) == 9
    d = glr_dims(batch=1, seqlen=200)
    cu = cu_array([0, 0, 1, 65, 130, 200, 200])
    assert lib.ssd_glr_chunk_rows(ctypes.byref(d), cu.ctypes.data, 6) == 1 + 1 + 2 + 2


@pytest.mark.parametrize("name", ["x", "r", "i", "A", "y"])
def test_glr_forward_pointers(lib, name):
    assert forward(lib, glr_dims(), **{name: None}) == NULL
    assert forward(lib, glr_dims(), **{name: FAKE + 8}) == MISALIGNED


@pytest.mark.parametrize("name", ["h0", "fin", "st"])
def test_glr_forward_optional_pointers(lib, name):
    assert forward(lib, glr_dims(), **{name: FAKE + 4}) == MISALIGNED


@pytest.mark.parametrize("name", ["x", "r", "i", "A", "st", "dy", "dx", "dr", "di", "dA"])
def test_glr_backward_pointers(lib, name):
    assert backward(lib, glr_dims(), **{name: None}) == NULL
    assert backward(lib, glr_dims(), **{name: FAKE + 8}) == MISALIGNED


def test_glr_checkpoints(lib):
    assert forward(lib, glr_dims(), pk=packed(codes=None)) == NULL
    assert forward(lib, glr_dims(), pk=packed(last=None)) == NULL
    assert forward(lib, glr_dims(), pk=packed(exps=FAKE + 1)) == MISALIGNED
    none = dict(x=None, r=None, i=None)
    assert backward(lib, glr_dims(), pk=packed(exps=None), **none) == NULL
    assert backward(lib, glr_dims(), pk=packed(codes=FAKE + 8), **none) == MISALIGNED
    assert backward(lib, glr_dims(), pk=packed()) == INVALID  # both kinds of inputs


@pytest.mark.parametrize("kw,code", [(dict(seqlen=2), INVALID)] + [c for c in BAD_GLR if "seqlen" not in c[0]], ids=str)
def test_glr_step(lib, kw, code):
    d = glr_dims(**{"seqlen": 1, **kw})
    assert lib.ssd_glr_step(ctypes.byref(d), *[FAKE] * 6, None) == code
    one = glr_dims(seqlen=1)
    for n in range(6):
        args = [FAKE] * 6
        args[n] = None
        assert lib.ssd_glr_step(ctypes.byref(one), *args, None) == NULL
        args[n] = FAKE + 2
        assert lib.ssd_glr_step(ctypes.byref(one), *args, None) == MISALIGNED


@pytest.mark.parametrize("rows,cols,dtype,code", [(0, 8, 0, INVALID), (8, 0, 0, INVALID), (-1, 8, 0, INVALID),
                                                  (8, 8, 2, UNSUPPORTED), ((1 << 33) + 1, 1, 0, UNSUPPORTED),
                                                  (1 << 20, 1 << 30, 1, UNSUPPORTED)])
def test_pack8(lib, rows, cols, dtype, code):
    ok = binding._Packed8(FAKE, FAKE)
    assert lib.ssd_pack8(rows, cols, dtype, FAKE, ctypes.byref(ok), None) == code
    assert lib.ssd_unpack8(rows, cols, dtype, ctypes.byref(ok), FAKE, None) == code


def test_pack8_pointers(lib):
    ok = binding._Packed8(FAKE, FAKE)
    assert lib.ssd_pack8(8, 8, 0, None, ctypes.byref(ok), None) == NULL
    assert lib.ssd_pack8(8, 8, 0, FAKE, None, None) == NULL
    assert lib.ssd_pack8(8, 8, 0, FAKE + 4, ctypes.byref(ok), None) == MISALIGNED
    for bad, code in ((binding._Packed8(None, FAKE), NULL), (binding._Packed8(FAKE, None), NULL),
                      (binding._Packed8(FAKE + 1, FAKE), MISALIGNED), (binding._Packed8(FAKE, FAKE + 1), MISALIGNED)):
        assert lib.ssd_pack8(8, 8, 0, FAKE, ctypes.byref(bad), None) == code
        assert lib.ssd_unpack8(8, 8, 0, ctypes.byref(bad), FAKE, None) == code


def rot_dims(**kw):
    d = dict(batch=2, seqlen=8, ngroups=2, dstate=64, rotary=32, B_batch_stride=1024, B_token_stride=128,
             C_batch_stride=1024, C_token_stride=128, dtype=1, interleaved=0, eps=1e-5, reserved=0)
    d.update(kw)
    return binding.RotateDims(**d)


@pytest.mark.parametrize("kw,code", [(dict(batch=0), INVALID), (dict(seqlen=-1), INVALID), (dict(ngroups=0), INVALID),
                                     (dict(dstate=0), INVALID), (dict(rotary=33), INVALID), (dict(rotary=66), INVALID),
                                     (dict(rotary=-2), INVALID), (dict(eps=0.0), INVALID),
                                     (dict(eps=float("nan")), INVALID), (dict(reserved=1), INVALID),
                                     (dict(dtype=3), UNSUPPORTED), (dict(dstate=257), UNSUPPORTED),
                                     (dict(batch=1 << 20, seqlen=1 << 12), UNSUPPORTED)], ids=str)
def test_norm_rotate_sizes(lib, kw, code):
    d = rot_dims(**kw)
    assert lib.ssd_norm_rotate(ctypes.byref(d), *[FAKE] * 8, None) == code
    assert lib.ssd_norm_rotate_backward(ctypes.byref(d), *[FAKE] * 12, None) == code


def test_norm_rotate_pointers(lib):
    d = rot_dims()
    for n, optional in ((0, 0), (1, 0), (2, 0), (3, 0), (4, 1), (5, 1), (6, 0), (7, 0)):
        args = [FAKE] * 8
        args[n] = FAKE + 1
        assert lib.ssd_norm_rotate(ctypes.byref(d), *args, None) == MISALIGNED
        if not optional:
            args[n] = None
            assert lib.ssd_norm_rotate(ctypes.byref(d), *args, None) == NULL
    for n in range(12):
        args = [FAKE] * 12
        args[n] = FAKE + 1
        assert lib.ssd_norm_rotate_backward(ctypes.byref(d), *args, None) == MISALIGNED
        if n not in (6, 7, 10, 11):
            args[n] = None
            assert lib.ssd_norm_rotate_backward(ctypes.byref(d), *args, None) == NULL


def test_binding_refuses_host_tensors_and_other_types():
    x = torch.zeros(2, 3, 4)
    for call in (lambda: binding.glr_forward(x, x, x, torch.zeros(4)),
                 lambda: binding.glr_step(x[:, 0], x[:, 0], x[:, 0], x[:, 0], torch.zeros(4)),
                 lambda: binding.pack8(x), lambda: binding.unpack8(x),
                 lambda: binding.unpack8(binding.Packed8(torch.zeros(2, 3, dtype=torch.int8),
                                                         torch.zeros(2, 1, dtype=torch.uint8))),
                 lambda: binding.glr_backward(x, None),
                 lambda: binding.norm_rotate(x[None], x[None], torch.zeros(1, 2, dtype=torch.int64), torch.zeros(2))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refusals_on_the_device():
    dev = "cuda:0"
    x, A = torch.zeros(2, 6, 8, device=dev), torch.zeros(8, device=dev)
    st = torch.zeros(2, 8, device=dev)
    ok = dict(x=x, r=x, i=x, A=A)

    def refuse(call, *a, **kw):
        with pytest.raises((ValueError, binding.SSDError)):
            call(*a, **kw)

    for kw in (dict(r=x[:, :5]), dict(i=x.bfloat16()), dict(A=A[:7]), dict(A=A.double()), dict(x=x.half()),
               dict(init_state=st[:1]), dict(init_state=st.bfloat16()), dict(cu_seqlens=[0, 6]),
               dict(save="8"), dict(out=x.bfloat16()), dict(x=x.transpose(1, 2)), dict(r=x.cpu()),
               dict(x=x[0]), dict(x=x[:0], r=x[:0], i=x[:0])):
        refuse(binding.glr_forward, **{**ok, **kw})
    one = {k: (v[:1] if v.dim() == 3 else v) for k, v in ok.items()}
    for cu in ([0, 5], [0, 4, 3, 6], [1, 6], [[0, 6]], [0]):
        refuse(binding.glr_forward, **one, cu_seqlens=cu)
    y, saved = binding.glr_forward(**ok, save="inputs")
    for dy in (x[:1], x.bfloat16(), x[..., :4].contiguous(), x.transpose(0, 1)):
        refuse(binding.glr_backward, dy, saved)
    refuse(binding.glr_backward, x, saved, dfinal_state=st[:1])
    refuse(binding.glr_backward, x, (x, x, x))
    refuse(binding.glr_step, st, x[:, 0], x[:, 0], x[:, 0], A)  # rows of a longer tensor
    refuse(binding.glr_step, st[:1], st, st, st, A)
    refuse(binding.glr_step, st.bfloat16(), st, st, st, A)
    refuse(binding.pack8, x.half())
    refuse(binding.pack8, x.transpose(1, 2))
    refuse(binding.pack8, x[..., :0])
    p = binding.pack8(x)
    refuse(binding.unpack8, p, torch.float16)
    refuse(binding.unpack8, binding.Packed8(p.codes, p.exps[:1]))
    refuse(binding.unpack8, binding.Packed8(p.codes.view(torch.uint8), p.exps))
    refuse(binding.unpack8, p, out=torch.zeros(2, 6, 8, device=dev))
    B, pos, f = torch.zeros(2, 3, 2, 8, device=dev), torch.zeros(2, 3, dtype=torch.int64, device=dev), A[:4]
    for a in ((B, B[:, :2], pos, f), (B, B.bfloat16(), pos, f), (B, B, pos.int(), f), (B, B, pos[0], f),
              (B, B, pos, torch.zeros(5, device=dev)), (B.transpose(2, 3), B.transpose(2, 3), pos, f),
              (B[..., ::2], B[..., ::2], pos, f[:2]), (B[0], B[0], pos, f)):
        refuse(binding.norm_rotate, *a)
    refuse(binding.norm_rotate, B, B, pos, f, weight_B=A[:4])
    refuse(binding.norm_rotate, B, B, pos, f, eps=0.0)
    refuse(binding.norm_rotate_backward, B[:, :2], B, B, B, pos, f)


def test_ssd_backward_packed8_refusals(lib):
    d = binding.make_dims(batch=1, seqlen=64, nheads=2, headdim=64, dstate=64, ngroups=1, dtype="bf16")

    def call(pk, chunk=64, **kw):
        p = [FAKE] * 3 + [chunk, None, FAKE, None] + [FAKE] * 6 + [None]  # dt A D | chunk h0 dy dfin | dx .. dD | dinit
        for k, v in kw.items():
            p[int(k[1:])] = v
        return lib.ssd_backward_packed8(ctypes.byref(d), pk, *p, None)

    assert call(None) == NULL
    assert call(packed(codes=None)) == NULL and call(packed(last=None)) == NULL
    assert call(packed(exps=FAKE + 1)) == MISALIGNED
    assert call(packed(), chunk=63) == UNSUPPORTED
    assert call(packed(), a0=None) == NULL and call(packed(), a5=None) == NULL
    assert call(packed(), a7=FAKE + 4) == MISALIGNED
