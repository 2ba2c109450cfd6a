"""Workloads of the gated linear recurrence, the 8-bit activation checkpoints and
the norm and rotation of B and C: inputs, plain forms, and what each has to
move.

A case's ``op`` says what one pass does:

  glr       the recurrence over whole sequences (prefill), batched or packed
  glr_step  one token of it for every row of a batch (decode), on a kept state
  glr_train its forward pass and its backward pass; with ``packed`` the inputs
            are kept as 8-bit checkpoints between the two
  pack      an activation into its 8-bit checkpoint and back
  rotate    RMSNorm over each group's state dimension and the position rotation
            of the scan's B and C
  rotate_train  that and its backward pass

``run`` computes the plain form with elementary torch operations, or, where
``own`` is true, makes the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 64  # values that share an exponent in a checkpoint
CHUNK = 64  # tokens between two states that the forward pass keeps


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _glr(name, op, batch, seqlen, channels, dtype, init=True, nseq=0, packed=False):
    return dict(name=name, op=op, batch=batch, seqlen=seqlen, channels=channels, dtype=dtype, init=init,
                nseq=nseq, packed=packed)


def _rot(name, op, batch, seqlen, ngroups, dstate, dtype, rotary, interleaved, slices, far):
    return dict(name=name, op=op, batch=batch, seqlen=seqlen, ngroups=ngroups, dstate=dstate, dtype=dtype,
                rotary=rotary, interleaved=interleaved, slices=slices, far=far)


def listed():
    return [
        # prefill of the layer with 80 heads of 64 values
        _glr("glr_prefill_80x64", "glr", 4, 4096, 5120, "bf16"),
        # one long sequence, 32 heads of 64 values
        _glr("glr_prefill_long", "glr", 1, 65536, 2048, "bf16", init=False),
        # prompts of many lengths (empty and one-token ones among them) packed along one row
        _glr("glr_packed_prompts_f32", "glr", 1, 8190, 1536, "f32", nseq=61),
        # one decode step of a serving batch
        _glr("glr_decode_64", "glr_step", 64, 1, 5120, "bf16"),
        # a training step of the layer with 24 heads of 64 values
        _glr("glr_train_24x64", "glr_train", 8, 2048, 1536, "bf16", init=False),
        # odd sizes in 32 bits, as in a test of gradients
        _glr("glr_train_odd_f32", "glr_train", 3, 1021, 333, "f32"),
        # the large layer's training step with its inputs kept in 8 bits
        _glr("glr_train_packed_80x64", "glr_train", 4, 4096, 5120, "bf16", init=False, packed=True),
        # one activation of that layer kept in 8 bits and read back
        dict(name="pack_80x64", op="pack", rows=16384, cols=5120, dtype="bf16"),
        # B and C of a long grouped prefill, slices of one projection
        _rot("rotate_prefill_long", "rotate", 1, 65536, 8, 128, "bf16", 128, False, True, False),
        # B and C of a decode step, far positions
        _rot("rotate_decode_64", "rotate", 64, 1, 8, 128, "bf16", 64, True, False, True),
        # training with one group
        _rot("rotate_train_g1", "rotate_train", 4, 4096, 1, 128, "bf16", 128, False, True, False),
        # training with groups in 32 bits, a state dimension off the powers of two
        _rot("rotate_train_g4_f32", "rotate_train", 2, 2047, 4, 96, "f32", 64, True, False, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glr", "glr", "glr_step", "glr_train", "glr_train", "pack", "rotate", "rotate_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "pack":
        cols = _log(rng, 16, 6144)
        return dict(op=op, rows=_log(rng, 1, max(2, 20_000_000 // cols)), cols=cols, dtype=dtype)
    if op.startswith("rotate"):
        dstate = 8 * rng.randint(2, 32)
        ngroups = rng.choice([1, 1, 2, 4, 5, 8])
        batch = _log(rng, 1, 64)
        seqlen = _log(rng, 1, max(2, min(65536, 12_000_000 // (batch * ngroups * dstate))))
        c = _rot("", op, batch, seqlen, ngroups, dstate, dtype, rng.choice([dstate, dstate // 8 * 4]),
                 rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5)
    else:
        channels = _log(rng, 16, 6144)
        if rng.random() < 0.6:
            channels = max(8, channels // 8 * 8)
        batch = _log(rng, 1, 16) if op != "glr_step" else _log(rng, 1, 256)
        nseq = _log(rng, 2, 300) if op != "glr_step" and rng.random() < 0.3 else 0
        if nseq:
            batch = 1
        most = 16_000_000 // (batch * channels)
        seqlen = 1 if op == "glr_step" else _log(rng, max(1, nseq), max(nseq + 2, min(65536, most)))
        c = _glr("", op, batch, seqlen, channels, dtype, rng.random() < 0.5, nseq,
                 op == "glr_train" and rng.random() < 0.5)
    del c["name"]
    return c


def offsets(case):
    """nseq + 1 offsets of the packed sequences (none: a plain batch); they
    belong to the case: empty and one-token sequences among them."""
    n, total = case["nseq"], case["seqlen"]
    if not n:
        return None
    rng = random.Random(n * 1009 + total)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    for j in range(1, len(cuts), 7):
        cuts[j] = cuts[j - 1]
    for j in range(4, len(cuts), 9):
        cuts[j] = min(cuts[j - 1] + 1, cuts[j])
    return [0] + cuts + [total]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, to=dtype):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(scale).add_(shift).to(to)

    s = dict(case=case)
    if case["op"] == "pack":
        # an activation after a norm, a few channels much larger than the rest
        x = torch.randn(case["rows"], case["cols"], generator=gen, device=DEV)
        x *= torch.exp(0.8 * torch.randn(case["cols"], generator=gen, device=DEV))
        s["x"] = x.to(dtype)
        return s
    b, t = case["batch"], case["seqlen"]
    if case["op"].startswith("rotate"):
        g, n = case["ngroups"], case["dstate"]
        if case["slices"]:
            # B and C as the scan's projection leaves them: side by side in one row
            both = normal(b, t, 2 * g * n, scale=2.0)
            s["B"] = both[..., : g * n].unflatten(-1, (g, n))
            s["C"] = both[..., g * n:].unflatten(-1, (g, n))
        else:
            s["B"], s["C"] = normal(b, t, g, n, scale=2.0), normal(b, t, g, n, scale=0.5)
        s["wB"] = normal(n, scale=0.2, shift=1.0, to=torch.float32)
        s["wC"] = normal(n, scale=0.2, shift=1.0, to=torch.float32)
        start = torch.randint(0, 900_000 if case["far"] else 4096, (b, 1), generator=gen, device=DEV)
        s["positions"] = start + torch.arange(t, device=DEV)
        half = case["rotary"] // 2
        s["inv_freq"] = torch.exp(-math.log(10000.0) * torch.arange(half, device=DEV, dtype=torch.float32) / half)
        if case["op"] == "rotate_train":
            s["dB"], s["dC"] = normal(b, t, g, n), normal(b, t, g, n)
        return s
    c = case["channels"]
    cu = offsets(case)
    s["cu"] = cu
    rows = case["nseq"] or b
    if case["op"] == "glr_step":
        s["x"], s["r"], s["i"] = normal(b, c), normal(b, c), normal(b, c)
        s["state"] = normal(b, c, to=torch.float32)
    else:
        s["x"], s["r"], s["i"] = normal(b, t, c), normal(b, t, c), normal(b, t, c)
        s["init"] = normal(rows, c, to=torch.float32) if case["init"] else None
    # decays of 0.9 to 0.999 a token with the gate open halfway
    base = 0.9 + 0.099 * torch.rand(c, generator=gen, device=DEV)
    s["A"] = 2.0 * torch.log(base)
    if case["op"] == "glr_train":
        s["dy"] = normal(b, t, c)
        s["dfinal"] = normal(rows, c, to=torch.float32) if case["init"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1, from zero, by doubling: in 64 bits,
    as long products of decays next to one lose too much in 32."""
    a, u = a.double(), u.double()
    shift, total = 1, a.shape[1]
    while shift < total:
        u = torch.cat([u[:, :shift], u[:, shift:] + a[:, shift:] * u[:, :-shift]], dim=1)
        a = torch.cat([a[:, :shift], a[:, shift:] * a[:, :-shift]], dim=1)
        shift *= 2
    return u.float()


def _ends(case, cu):
    """(batch row, first token, last token + 1) of each sequence, as index tensors."""
    if cu is None:
        b = torch.arange(case["batch"], device=DEV)
        return b, torch.zeros_like(b), torch.full_like(b, case["seqlen"])
    at = torch.tensor(cu, device=DEV)
    return torch.zeros_like(at[1:]), at[:-1], at[1:]


def _gates(x, r, i, A):
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    la = A * sr
    a = torch.exp(la.double())  # a decay next to one, taken many times over
    v = -torch.expm1(2 * la)
    m = torch.sqrt(v)
    return sr, si, la, a, m, m * si * x


def _states(a, u, case, cu, init):
    """h, with each sequence's own start, and the state after each sequence."""
    row, lo, hi = _ends(case, cu)
    some = hi > lo
    a, u = a.clone(), u.double()
    if init is not None:
        u[row[some], lo[some]] += a[row[some], lo[some]] * init[some]
    a[row[some], lo[some]] = 0
    h = _scan(a, u)
    final = torch.zeros(len(lo), a.shape[2], device=DEV) if init is None else init.clone()
    final[some] = h[row[some], hi[some] - 1]
    return h, final


def _before(h, case, cu, init):
    """The state before each token."""
    row, lo, hi = _ends(case, cu)
    some = hi > lo
    p = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], dim=1)
    p[row[some], lo[some]] = 0 if init is None else init[some]
    return p


def _chunk_starts(case, cu):
    """Whether a token is the first of a chunk of its sequence, [batch, seqlen]."""
    t = torch.arange(case["seqlen"], device=DEV)
    if cu is None:
        return (t % CHUNK == 0).expand(case["batch"], -1)
    at = torch.tensor(cu, device=DEV)
    first = at[torch.searchsorted(at, t, right=True) - 1]
    return ((t - first) % CHUNK == 0)[None]


def _pack(x):
    """x as its 8-bit checkpoint holds it, in 32 bits: blocks along the last
    dimension, codes of one byte times a power of two, the smallest with which
    the block's largest magnitude rounds to 127 or less."""
    c = x.shape[-1]
    blocks = torch.nn.functional.pad(x.float(), (0, -c % BLOCK)).unflatten(-1, (-1, BLOCK))
    m, k = torch.frexp(blocks.abs().amax(-1, keepdim=True))
    e = torch.where(m < 127.5 / 128, k - 7, k - 6).clamp(min=-126)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    # 2^e and 2^-e by their bits: a rounded power would move values off ties
    up, down = ((e + 127) << 23).view(torch.float32), ((127 - e) << 23).view(torch.float32)
    return (torch.round(blocks * down) * up).flatten(-2)[..., :c]


def _glr_plain(s):
    case, cu, init = s["case"], s["cu"], s["init"]
    dtype = TYPES[case["dtype"]]
    x, r, i, A = s["x"].float(), s["r"].float(), s["i"].float(), s["A"]
    _, _, _, a, _, u = _gates(x, r, i, A)
    h, final = _states(a, u, case, cu, init)
    out = dict(y=h.to(dtype), final=final)
    if case["op"] == "glr":
        return out
    before = _before(h, case, cu, init)
    if case["packed"]:
        x, r, i = _pack(x), _pack(r), _pack(i)
    sr, si, la, a, m, u = _gates(x, r, i, A)
    if case["packed"]:
        # the states inside a chunk, from the kept one before it
        start = _chunk_starts(case, cu)[..., None]
        h = _scan(torch.where(start, torch.zeros_like(a), a), torch.where(start, u + a * before, u))
        before = torch.where(start, before, torch.cat([h[:, :1], h[:, :-1]], dim=1))
    row, lo, hi = _ends(case, cu)
    some = hi > lo
    g = s["dy"].float().clone()
    nexta = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], dim=1)
    nexta[row[some], hi[some] - 1] = 0
    if s["dfinal"] is not None:
        g[row[some], hi[some] - 1] += s["dfinal"][some]
    G = _scan(nexta.flip(1), g.flip(1)).flip(1)
    dla = G * (a * before - torch.where(m > 0, a * a * si * x / m, torch.zeros_like(m)))
    out["dx"] = (G * m * si).to(dtype)
    out["dr"] = (dla * la * torch.sigmoid(-r)).to(dtype)
    out["di"] = (G * u * torch.sigmoid(-i)).to(dtype)
    out["dA"] = (dla * sr).sum((0, 1)).float()
    if init is not None:
        out["dinit"] = torch.zeros_like(init) if s["dfinal"] is None else s["dfinal"].clone()
        out["dinit"][some] = (a[row[some], lo[some]] * G[row[some], lo[some]]).float()
    return out


def _turn(z, cos, sin, half, interleaved):
    """Rotates the first 2 * half values of z's last dimension by pairs."""
    head, rest = z[..., : 2 * half], z[..., 2 * half:]
    if interleaved:
        p, q = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([p * cos - q * sin, p * sin + q * cos], dim=-1).flatten(-2), rest], dim=-1)
    p, q = head[..., :half], head[..., half:]
    return torch.cat([p * cos - q * sin, p * sin + q * cos, rest], dim=-1)


def _rotate_plain(s):
    case = s["case"]
    dtype, half, inter = TYPES[case["dtype"]], case["rotary"] // 2, case["interleaved"]
    angle = s["positions"].double()[..., None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[..., None, :], angle.sin().float()[..., None, :]
    out = {}
    for k in ("B", "C"):
        x, w = s[k].float(), s["w" + k]
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
        xh = x * rstd
        out[k] = _turn(xh * w, cos, sin, half, inter).to(dtype)
        if case["op"] == "rotate_train":
            dz = _turn(s["d" + k].float(), cos, -sin, half, inter)
            out["dw" + k] = (dz * xh).sum((0, 1, 2))
            dxh = dz * w
            out["d" + k] = (rstd * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))).to(dtype)
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _run_own(s):
    from structured_state_space_mamba_b200 import binding
    case, op = s["case"], s["case"]["op"]
    if op == "pack":
        return binding.unpack8(binding.pack8(s["x"]), s["x"].dtype)
    if op == "glr_step":
        y = binding.glr_step(s["state"], s["x"], s["r"], s["i"], s["A"])
        return dict(y=y, state=s["state"])
    if op == "glr":
        y, final = binding.glr_forward(s["x"], s["r"], s["i"], s["A"], init_state=s["init"], cu_seqlens=s["cu"],
                                       return_final_state=True)
        return dict(y=y, final=final)
    if op == "glr_train":
        y, final, saved = binding.glr_forward(s["x"], s["r"], s["i"], s["A"], init_state=s["init"],
                                              cu_seqlens=s["cu"], return_final_state=True,
                                              save="packed8" if case["packed"] else "inputs")
        g = binding.glr_backward(s["dy"], saved, dfinal_state=s["dfinal"], return_dinit_state=case["init"])
        out = dict(y=y, final=final, dx=g["dx"], dr=g["dr"], di=g["di"], dA=g["dA"])
        if case["init"]:
            out["dinit"] = g["dinit_state"]
        return out
    kw = dict(weight_B=s["wB"], weight_C=s["wC"], eps=1e-5, interleaved=case["interleaved"])
    B, C = binding.norm_rotate(s["B"], s["C"], s["positions"], s["inv_freq"], **kw)
    if op == "rotate":
        return dict(B=B, C=C)
    g = binding.norm_rotate_backward(s["dB"], s["dC"], s["B"], s["C"], s["positions"], s["inv_freq"], **kw)
    return dict(B=B, C=C, dB=g["dB"], dC=g["dC"], dwB=g["dweight_B"], dwC=g["dweight_C"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "pack":
        return _pack(state["x"]).to(state["x"].dtype)
    if op == "glr_step":
        _, _, _, a, _, u = _gates(state["x"].float(), state["r"].float(), state["i"].float(), state["A"])
        state["state"].copy_(state["state"] * a + u)
        return dict(y=state["state"].to(state["x"].dtype), state=state["state"])
    return _rotate_plain(state) if op.startswith("rotate") else _glr_plain(state)


def work(case):
    """Inputs read once, outputs written once; arithmetic a value counted from
    the formulas, a special function as one."""
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "pack":
        n = case["rows"] * case["cols"]
        # the activation in, the checkpoint and the values that it stands for out
        return dict(bytes=n * (2 * es + 1) + case["rows"] * -(-case["cols"] // BLOCK), flops=4 * n)
    if case["op"].startswith("rotate"):
        tokens = case["batch"] * case["seqlen"]
        n = tokens * case["ngroups"] * case["dstate"]  # values of B, and of C
        small = 8 * tokens + 4 * (case["rotary"] // 2 + 2 * case["dstate"])
        if case["op"] == "rotate":
            return dict(bytes=4 * n * es + small, flops=2 * n * 7)
        return dict(bytes=8 * n * es + small + 8 * case["dstate"], flops=2 * n * 20)
    rows, c = case["nseq"] or case["batch"], case["channels"]
    n = case["batch"] * case["seqlen"] * c
    if case["op"] == "glr_step":
        return dict(bytes=4 * n * es + 8 * n + 4 * c, flops=14 * n)
    small = 4 * c + 4 * rows * c * (2 if case["init"] else 1)
    if case["op"] == "glr":
        return dict(bytes=4 * n * es + small, flops=14 * n)
    return dict(bytes=8 * n * es + small + 4 * c + (8 * rows * c if case["init"] else 0), flops=50 * n)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_pack(x):
    """Block by block: the exponent is the least whole e >= -126 with
    max|x| < 127.5 * 2^e."""
    x = x.double()
    out = torch.empty_like(x)
    for lo in range(0, x.shape[-1], BLOCK):
        part = x[..., lo: lo + BLOCK]
        top = part.abs().max(-1, keepdim=True).values
        step = torch.full_like(top, 2.0 ** -126)
        e = torch.log2(top.clamp(min=1e-300) / 127.5).floor().clamp(min=-126)
        for near in (1.0, 0.0, -1.0):  # the last one that holds is the least
            # the power of two by its bits
            trial = ((((e + near).clamp(min=-126)).long() + 1023) << 52).view(torch.float64)
            step = torch.where(top < 127.5 * trial, trial, step)
        out[..., lo: lo + BLOCK] = torch.round(part / step) * step
    return out


def _exact_glr(s):
    case, cu = s["case"], s["cu"]
    init, A = s["init"], s["A"].double()
    x, r, i = s["x"].double(), s["r"].double(), s["i"].double()
    B, T, C = x.shape
    rows = case["nseq"] or B
    start = torch.zeros(rows, C, dtype=torch.float64, device=DEV) if init is None else init.double()
    # sequences that begin at a token, and those that end with it
    begins, ends = {}, {}
    if cu is None:
        begins[0], ends[T - 1] = slice(0, B), slice(0, B)
    else:
        for j in range(case["nseq"]):
            if cu[j + 1] > cu[j]:
                begins[cu[j]] = ends[cu[j + 1] - 1] = slice(j, j + 1)

    def coefficients(r, i, x):
        gate = 1 / (1 + torch.exp(-r))
        decay = torch.exp(A * gate)
        root = torch.sqrt(1 - decay * decay)
        return gate, decay, root, 1 / (1 + torch.exp(-i))

    gate, decay, root, inp = coefficients(r, i, x)
    y = torch.empty_like(x)
    prev = torch.empty_like(x)  # the state before each token
    final = start.clone()
    h = start[:B]
    for t in range(T):
        if t in begins:
            h = start[begins[t]]
        prev[:, t] = h
        h = decay[:, t] * h + root[:, t] * inp[:, t] * x[:, t]
        y[:, t] = h
        if t in ends:
            final[ends[t]] = h
    out = dict(y=y, final=final)
    if case["op"] == "glr":
        return out
    if case["packed"]:
        x, r, i = _exact_pack(x), _exact_pack(r), _exact_pack(i)
        gate, decay, root, inp = coefficients(r, i, x)
        since = 0
        for t in range(T):
            since = 0 if t in begins else since + 1
            if since % CHUNK:  # the others keep the forward pass's state
                prev[:, t] = decay[:, t - 1] * prev[:, t - 1] + root[:, t - 1] * inp[:, t - 1] * x[:, t - 1]
    dy = s["dy"].double()
    dfinal = torch.zeros_like(start) if s["dfinal"] is None else s["dfinal"].double()
    dinit = dfinal.clone()
    G = torch.empty_like(dy)
    carry = torch.zeros_like(dy[:, 0])
    for t in reversed(range(T)):
        if t in ends:
            carry = dfinal[ends[t]]
        G[:, t] = dy[:, t] + carry
        carry = decay[:, t] * G[:, t]
        if t in begins:
            dinit[begins[t]] = carry
    # d decay / d(A gate) = decay, d root / d(A gate) = -decay^2 / root
    dla = G * (decay * prev - torch.where(root > 0, decay * decay * inp * x / root, 0.0))
    out["dx"] = G * root * inp
    out["dr"] = dla * A * gate * (1 - gate)
    out["di"] = G * root * x * inp * (1 - inp)
    out["dA"] = torch.einsum("btc,btc->c", dla, gate)
    if init is not None:
        out["dinit"] = dinit
    return out


def _exact_rotate(s):
    case = s["case"]
    half, n = case["rotary"] // 2, case["dstate"]
    if case["interleaved"]:
        first = torch.arange(half, device=DEV) * 2
        second = first + 1
    else:
        first = torch.arange(half, device=DEV)
        second = first + half
    # each pair as a complex number, turned by e^(i angle)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.einsum("bt,k->btk", s["positions"].double(), s["inv_freq"].double()))[:, :, None]

    def turned(z, by):
        p = torch.complex(z[..., first], z[..., second]) * by
        o = z.clone()
        o[..., first], o[..., second] = p.real, p.imag
        return o

    out = {}
    for k in ("B", "C"):
        x, w = s[k].double(), s["w" + k].double()
        size = torch.sqrt((x.square().sum(-1, keepdim=True) / n) + 1e-5)
        out[k] = turned(x / size * w, turn)
        if case["op"] == "rotate_train":
            dz = turned(s["d" + k].double(), turn.conj())
            out["dw" + k] = torch.einsum("btgn,btgn->n", dz, x / size)
            d = dz * w
            out["d" + k] = d / size - x * (d * x).sum(-1, keepdim=True) / (n * size ** 3)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pack":
        return _exact_pack(s["x"])
    if case["op"] == "glr_step":
        g, k = 1 / (1 + torch.exp(-s["r"].double())), 1 / (1 + torch.exp(-s["i"].double()))
        decay = torch.exp(s["A"].double() * g)
        h = decay * s["state"].double() + torch.sqrt(1 - decay ** 2) * k * s["x"].double()
        return dict(y=h, state=h)
    return _exact_rotate(s) if case["op"].startswith("rotate") else _exact_glr(s)
