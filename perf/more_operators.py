"""More operators around one MoE layer: what is computed, on which sizes, and
their plain forms.

Operators:

  quant4     a matrix in 4-bit blocks (e2m1 codes, 32 of them to a power-of-two
             scale), and its values back;
  experts4   the routed experts' SwiGLU block on 4-bit weights and 8-bit rows
             (dispatch, both products, gate-weighted combine);
  few        the whole layer for a few tokens: router, top-k, experts, shared
             expert, combine, on bfloat16, 8-bit or 4-bit weights;
  step       what lies between two blocks of a residual stream: the norm behind
             a block, its gate, the residual's scale and addition, and the norm
             in front of the next block;
  step_bwd   its backward.

``own`` False computes them with elementary torch operations in float32; True
calls the library. ``exact`` computes them in float64.

4-bit blocks: 32 consecutive values of a row share the scale 2^e, e the
smallest integer >= -127 with max|v| <= 6 * 2^e (6 is e2m1's largest value, so
nothing saturates); the codes are v / 2^e rounded to nearest even among 0, 1/2,
1, 3/2, 2, 3, 4, 6 and their negatives, value 2i in the low half of byte i. The
scale is stored as the byte e + 127. 8-bit blocks have e4m3 codes and 448 in the
place of 6.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}
BLOCK = 32
MX8, MX4 = "mx8", "mx4"


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # rows of a float32 model, an odd number of them: launches count
        dict(name="quant4_f32_1021", op="quant4", rows=1021, cols=2080, dtype=F32),
        # one projection of 128 experts when a model is loaded
        dict(name="quant4_experts", op="quant4", rows=128 * 1536, cols=4096, dtype=BF16),
        # a decode batch: every expert with a few rows, the weights' stream counts
        dict(name="experts4_decode_256", op="experts4", T=256, H=4096, E=128, k=8, F=1536, R=16, skew=0.2),
        # few wide experts, a ragged token count: bound by the matrix cores
        dict(name="experts4_mixtral_2047", op="experts4", T=2047, H=4096, E=8, k=2, F=14336, R=8, skew=0.1),
        # the largest layer: 65536 rows against 256 experts
        dict(name="experts4_dsv3_8192", op="experts4", T=8192, H=7168, E=256, k=8, F=2048, R=32, skew=0.2),
        # decoding one token with bfloat16 weights: latency, and 8 experts' weights
        dict(name="few_bf16_1", op="few", T=1, H=4096, E=128, k=8, F=1536, shared_F=0, weights=BF16),
        # five sequences on few wide experts in 8 bits
        dict(name="few_mx8_5", op="few", T=5, H=4096, E=8, k=2, F=14336, shared_F=0, weights=MX8),
        # sixteen sequences of the largest layer in 4 bits, with its shared expert
        dict(name="few_mx4_16", op="few", T=16, H=7168, E=256, k=8, F=2048, shared_F=2048, weights=MX4),
        # between two blocks of one decoded token: latency
        dict(name="step_decode_1", op="step", T=1, H=4096, dtype=BF16, gate="channel", rows=1, mx=True),
        # a prefill batch; every token has its own gate
        dict(name="step_prefill_8192", op="step", T=8192, H=7168, dtype=BF16, gate="token", rows=1, mx=True),
        # training, the widest batch, one gate for each channel
        dict(name="step_bwd_8192", op="step_bwd", T=8192, H=7168, dtype=BF16, gate="channel", rows=8192),
        # training a small float32 model: a row of gates for every 37 tokens
        dict(name="step_bwd_f32_777", op="step_bwd", T=777, H=1540, dtype=F32, gate="channel", rows=37),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant4", "experts4", "experts4", "few", "few", "step", "step_bwd"])
    if op == "quant4":
        cols = _log(rng, 1, 448) * BLOCK
        return dict(op=op, rows=_log(rng, 1, min(1 << 20, 800_000_000 // cols)), cols=cols, dtype=rng.choice([BF16, F32]))
    if op == "experts4":
        while True:
            E = rng.choice([4, 6, 8, 16, 40, 64, 96, 128, 256])
            R = rng.choice([r for r in range(1, 33) if E % r == 0])
            k = rng.randint(1, min(8, E))
            H = _log(rng, 128, 7168) // 128 * 128
            F = _log(rng, 128, 8192) // 128 * 128
            T = _log(rng, 1, 8192)
            if E * 3 * F * H <= 4 << 30 and T * k * 6 * F * H <= 4e12:
                return dict(op=op, T=T, H=H, E=E, k=k, F=F, R=R, skew=round(rng.uniform(0, 0.6), 2))
    if op == "few":
        while True:
            E = rng.choice([4, 6, 8, 16, 40, 64, 96, 128, 256])
            k = rng.randint(1, min(8, E))
            H = _log(rng, 128, 7168) // 128 * 128
            F = _log(rng, 128, 8192) // 128 * 128
            T = rng.choice([1, 2, 3, 4, 6, 8, 11, 16, 24, 32])
            if E * 3 * F * H <= 2 << 30 and T * k * F * H <= 1.8e9:
                return dict(op=op, T=T, H=H, E=E, k=k, F=F, shared_F=rng.choice([0, 0, _log(rng, 128, 4096) // 128 * 128]),
                            weights=rng.choice([BF16, MX8, MX4]))
    dtype = rng.choice([BF16, BF16, F32])
    step = 64 if dtype == BF16 else 32
    T, H = _log(rng, 1, 8192), max(1, _log(rng, 64, 8192) // step) * step
    while T * H > 8192 * 7168 // (1 if dtype == BF16 else 2):
        T = T // 2 + 1
    c = dict(op=op, T=T, H=H, dtype=dtype, gate=rng.choice(["none", "token", "channel", "channel"]))
    c["rows"] = rng.choice([1, T, _log(rng, 1, T)])
    if op == "step":
        c["mx"] = rng.random() < 0.6
    return c


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1_000_003 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _channels(g, H):
    """Per-channel spread of a residual stream: most near 1, a few 10 and more."""
    return torch.exp(_randn(g, H) * 0.5) * (1 + 15 * (torch.rand(H, generator=g, device=DEV) < 0.004))


def _split(v, largest):
    """(v cut into blocks, exponents): the smallest e >= -127 with max|v| <=
    largest * 2^e. largest is 448 = 1.75 * 2^8 or 6 = 1.5 * 2^2."""
    b = v.view(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)
    top = b.abs().amax(-1)
    m, x = torch.frexp(top)
    over, place = (0.875, 9) if largest == 448 else (0.75, 3)
    e = x - place + (m > over).to(torch.int32)
    return b, torch.where(top == 0, torch.full_like(e, -127), e.clamp(min=-127))


def _bytes(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _pack8(v):
    """(e4m3 codes, scales) of float32 rows."""
    b, e = _split(v, 448)
    return torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(v.shape), _bytes(e)


def _e2m1(r):
    """Quotients up to 6 to the nearest e2m1 value, ties to even."""
    a = r.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(r / step) * step


def _pack4(v):
    """(bytes of two e2m1 codes, scales) of float32 rows."""
    b, e = _split(v, 6)
    r = _e2m1(torch.ldexp(b, -e.unsqueeze(-1))).view(v.shape)
    a = r.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a * 0.5 + 4)).to(torch.uint8) | (torch.signbit(r).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), _bytes(e)


def _weights(g, form, E, rows, cols):
    """A projection of E experts: (values, None) in bfloat16, or (codes, scales)."""
    wide = {BF16: (cols, torch.bfloat16), MX8: (cols, torch.float8_e4m3fn), MX4: (cols // 2, torch.uint8)}[form]
    q = torch.empty((E, rows, wide[0]), dtype=wide[1], device=DEV)
    s = None if form == BF16 else torch.empty((E, rows, cols // BLOCK), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (rows * cols))
    for a in range(0, E, step):
        b = min(E, a + step)
        v = _randn(g, b - a, rows, cols) / math.sqrt(cols)
        if form == BF16:
            q[a:b] = v.bfloat16()
        else:
            qa, sa = _pack8(v) if form == MX8 else _pack4(v)
            q[a:b].view(torch.uint8).copy_(qa.view(torch.uint8))
            s[a:b].copy_(sa.view(torch.uint8))
    return (q, None) if form == BF16 else (q, s.view(torch.float8_e8m0fnu))


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    st = {"case": c}
    if c["op"] == "quant4":
        t = _TYPES[c["dtype"]]
        st["x"] = torch.empty((c["rows"], c["cols"]), dtype=t, device=DEV)
        ch = _channels(g, c["cols"]) / math.sqrt(c["cols"])
        step = max(1, (1 << 27) // c["cols"])
        for a in range(0, c["rows"], step):
            b = min(c["rows"], a + step)
            st["x"][a:b] = _randn(g, b - a, c["cols"]) * ch
    elif c["op"] == "experts4":
        T, H, E, k, F = c["T"], c["H"], c["E"], c["k"], c["F"]
        x = _randn(g, T, H) * _channels(g, H)
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True))
        st["xq"], st["xs"] = _pack8(x)
        rank = torch.randperm(E, generator=g, device=DEV).float()
        logits = _randn(g, T, E)
        ids = torch.topk(logits - c["skew"] * torch.log1p(rank), k, dim=-1).indices
        st["w"] = torch.softmax(torch.gather(logits, 1, ids), -1)
        st["ids"] = ids.to(torch.int32)
        st["gate"], st["up"], st["down"] = (_weights(g, MX4, E, *s) for s in ((F, H), (F, H), (H, F)))
        # the plain form's padding: experts with rows, and the most rows of one
        counts = torch.bincount(ids.reshape(-1), minlength=E)
        st["live"] = counts.nonzero().reshape(-1)
        st["most"] = int(counts.max())
    elif c["op"] == "few":
        T, H, E, F, SF, form = c["T"], c["H"], c["E"], c["F"], c["shared_F"], c["weights"]
        x = _randn(g, T, H) * _channels(g, H)
        st["x"] = (x * torch.rsqrt(x.square().mean(-1, keepdim=True))).bfloat16()
        st["router"] = (_randn(g, E, H) * (1.5 / math.sqrt(H))).bfloat16()
        st["bias"] = _randn(g, E) * 0.1
        st["gate"], st["up"], st["down"] = (_weights(g, form, E, *s) for s in ((F, H), (F, H), (H, F)))
        st["shared"] = tuple(_weights(g, form, 1, *s) for s in ((SF, H), (SF, H), (H, SF))) if SF else None
    else:
        T, H, t = c["T"], c["H"], _TYPES[c["dtype"]]
        ch = _channels(g, H)
        st["x"] = (_randn(g, T, H) * ch * 0.3).to(t)
        st["residual"] = (_randn(g, T, H) * ch).to(t)
        st["w_post"] = (1 + 0.2 * _randn(g, H)).to(t)
        st["w_pre"] = (1 + 0.2 * _randn(g, H)).to(t)
        n = -(-T // c["rows"])
        st["gate"] = {"none": None, "token": torch.sigmoid(_randn(g, T)),
                      "channel": 0.5 + 0.2 * _randn(g, n, H)}[c["gate"]]
        if st["gate"] is not None:
            st["gate"] = st["gate"].to(t)
        st["alpha"] = 0.9
        if c["op"] == "step_bwd":
            # what the forward kept
            x = st["x"].double()
            st["rstd_post"] = torch.rsqrt(x.square().mean(-1) + EPS).float()
            y = x * st["rstd_post"].double().unsqueeze(-1) * st["w_post"].double()
            s = (0.9 * st["residual"].double() + y * (1.0 if st["gate"] is None else _rows(st, torch.float64))).to(t)
            st["s"] = s
            st["rstd_pre"] = torch.rsqrt(s.double().square().mean(-1) + EPS).float()
            st["dy"] = _randn(g, T, H).to(t)
            st["ds"] = _randn(g, T, H).to(t)
    return st


def _rows(st, t):
    """The gate as it multiplies rows: [T, 1], or [T, H] with a row for every `rows` tokens."""
    c, gate = st["case"], st["gate"].to(t)
    return gate.unsqueeze(-1) if c["gate"] == "token" else gate.repeat_interleave(c["rows"], 0)[:c["T"]]


# --------------------------------------------------------------- one pass ----

def run(state):
    return _RUN[state["case"]["op"]][1 if own else 0](state)


def _quant4_plain(st):
    b, e = _split(st["x"].float(), 6)
    e1 = e.unsqueeze(-1)
    v = torch.ldexp(_e2m1(torch.ldexp(b, -e1)), e1).view(st["x"].shape)
    return {"values": v.bfloat16(), "scales": _bytes(e)}


def _quant4_own(st):
    import expert_load_balance_amd as moe

    c = st["case"]
    q = torch.empty((c["rows"], c["cols"] // 2), dtype=torch.uint8, device=DEV)
    s = torch.empty((c["rows"], c["cols"] // BLOCK), dtype=torch.float8_e8m0fnu, device=DEV)
    v = torch.empty((c["rows"], c["cols"]), dtype=torch.bfloat16, device=DEV)
    moe.moe_mx4_quantize(st["x"], q, s)
    moe.moe_mx4_dequantize(q, s, v)
    return {"values": v, "scales": s}


def _values8(q, s):
    """float32 values of 8-bit blocks."""
    return (q.float().view(*s.shape, BLOCK) * s.float().unsqueeze(-1)).view(q.shape)


def _values4(q, s):
    """float32 values of 4-bit blocks."""
    c = torch.stack((q & 15, q >> 4), -1)
    a = (c & 7).float()
    a = torch.where(a < 4, a * 0.5, torch.where(a < 6, a - 2, a * 2 - 8))
    a = torch.where(c > 7, -a, a)
    return (a.view(*s.shape, BLOCK) * s.float().unsqueeze(-1)).view(*s.shape[:-1], s.shape[-1] * BLOCK)


def _bytes_at(t, i):
    """Rows i of an 8-bit tensor."""
    return t.view(torch.uint8)[i].view(t.dtype)


def _experts4_plain(st):
    c = st["case"]
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    live, most = st["live"], st["most"]
    flat = st["ids"].reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    by = flat[order]
    counts = torch.zeros(E, dtype=torch.long, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    place = torch.arange(T * k, device=DEV) - (torch.cumsum(counts, 0) - counts)[by]
    slot = torch.searchsorted(live, by)
    rows = torch.zeros((live.numel(), most, H), device=DEV)
    rows[slot, place] = _values8(st["xq"], st["xs"])[order // k]

    def times(a, w):
        return torch.bmm(a, _values4(w[0][live], _bytes_at(w[1], live)).transpose(1, 2))

    g = times(rows, st["gate"])
    h = g * torch.sigmoid(g) * times(rows, st["up"])
    y = times(_values8(*_pack8(h)), st["down"])[slot, place]
    per = torch.empty((T * k, H), device=DEV)
    per[order] = y
    return {"out": (per.view(T, k, H) * st["w"].unsqueeze(-1)).sum(1).to(torch.bfloat16)}


def _experts4_own(st):
    import expert_load_balance_amd as moe

    c = st["case"]
    if "layer" not in st:  # buffers and workspace that a program keeps per shape
        from expert_load_balance_amd.layer import MoeLayerMx

        st["layer"] = MoeLayerMx(moe.Shape(c["T"], c["H"], c["E"], c["k"], c["F"], c["R"], 0, moe.MOE_BF16), DEV,
                                 weight_bits=4)
    return {"out": st["layer"].experts(st["xq"], st["xs"], st["ids"], st["w"], st["gate"], st["up"], st["down"])}


def _picked(w, form, ids):
    """float32 values of the experts `ids` of a projection."""
    if form == BF16:
        return w[0][ids].float()
    return (_values8 if form == MX8 else _values4)(_bytes_at(w[0], ids), _bytes_at(w[1], ids))


def _few_plain(st):
    c = st["case"]
    T, H, k, form = c["T"], c["H"], c["k"], c["weights"]
    x = st["x"].float()
    logits = x @ st["router"].float().t()
    ids = torch.sort(logits + st["bias"], dim=-1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(logits, 1, ids)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    flat = ids.reshape(-1)
    rows = x.repeat_interleave(k, 0).unsqueeze(-1)
    g = torch.bmm(_picked(st["gate"], form, flat), rows)
    h = g * torch.sigmoid(g) * torch.bmm(_picked(st["up"], form, flat), rows)
    y = torch.bmm(_picked(st["down"], form, flat), h).view(T, k, H)
    out = (y * w.unsqueeze(-1)).sum(1)
    if st["shared"] is not None:
        one = torch.zeros(1, dtype=torch.long, device=DEV)
        sg, su, sd = (_picked(m, form, one)[0] for m in st["shared"])
        g = x @ sg.t()
        out = out + (g * torch.sigmoid(g) * (x @ su.t())) @ sd.t()
    return {"out": out.to(torch.bfloat16)}


def _few_own(st):
    import expert_load_balance_amd as moe

    c = st["case"]
    if "layer" not in st:  # buffers and workspace that a program keeps per shape
        from expert_load_balance_amd.layer import MoeLayerFew

        st["layer"] = MoeLayerFew(moe.Shape(c["T"], c["H"], c["E"], c["k"], c["F"], 1, 0, moe.MOE_BF16), DEV,
                                  weights=c["weights"], shared_F=c["shared_F"] or None)
    return {"out": st["layer"].forward(st["x"], st["router"], st["bias"], st["gate"], st["up"], st["down"], st["shared"])}


def _step_plain(st):
    c, t = st["case"], _TYPES[st["case"]["dtype"]]
    x = st["x"].float()
    r1 = torch.rsqrt(x.square().mean(-1) + EPS)
    n = x * r1.unsqueeze(-1) * st["w_post"].float()
    if st["gate"] is not None:
        n = n * _rows(st, torch.float32)
    s = (st["alpha"] * st["residual"].float() + n).to(t)
    sf = s.float()
    r2 = torch.rsqrt(sf.square().mean(-1) + EPS)
    y = sf * r2.unsqueeze(-1) * st["w_pre"].float()
    out = {"s": s, "y": y.to(t), "rstd_post": r1, "rstd_pre": r2}
    if c["mx"]:
        out["q"], out["scales"] = _pack8(y)
    return out


def _step_shape(moe, c):
    return moe.Shape(c["T"], c["H"], 1, 1, 64, 1, 0, moe.MOE_BF16 if c["dtype"] == BF16 else moe.MOE_F32)


def _gate_rows(c):
    """The library's layout of the gate: 0 for one value a token, else tokens to a row of gates."""
    return 0 if c["gate"] != "channel" else c["rows"]


def _step_own(st):
    import expert_load_balance_amd as moe

    c, x = st["case"], st["x"]
    T, H = c["T"], c["H"]
    out = {"s": torch.empty_like(x), "y": torch.empty_like(x), "rstd_post": torch.empty(T, device=DEV),
           "rstd_pre": torch.empty(T, device=DEV)}
    if c["mx"]:
        out["q"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
        out["scales"] = torch.empty((T, H // BLOCK), dtype=torch.float8_e8m0fnu, device=DEV)
    moe.moe_block_norm(_step_shape(moe, c), x, EPS, residual=st["residual"], alpha=st["alpha"], w_post=st["w_post"],
                       gate=st["gate"], gate_rows=_gate_rows(c), w_pre=st["w_pre"], s=out["s"], y=out["y"],
                       q=out.get("q"), scales=out.get("scales"), rstd_post=out["rstd_post"], rstd_pre=out["rstd_pre"])
    return out


def _step_bwd_plain(st):
    c, t = st["case"], _TYPES[st["case"]["dtype"]]
    r1, r2 = st["rstd_post"].unsqueeze(-1), st["rstd_pre"].unsqueeze(-1)
    sh, xh, dy = st["s"].float() * r2, st["x"].float() * r1, st["dy"].float()
    gw = dy * st["w_pre"].float()
    d = (gw - sh * (gw * sh).mean(-1, keepdim=True)) * r2 + st["ds"].float()
    dn = d if st["gate"] is None else d * _rows(st, torch.float32)
    gw = dn * st["w_post"].float()
    dx = (gw - xh * (gw * xh).mean(-1, keepdim=True)) * r1
    out = {"dx": dx.to(t), "dresidual": (st["alpha"] * d).to(t), "dw_post": (dn * xh).sum(0), "dw_pre": (dy * sh).sum(0)}
    if st["gate"] is not None:
        p = d * xh * st["w_post"].float()
        if c["gate"] == "token":
            out["dgate"] = p.sum(-1)
        else:
            at = torch.arange(c["T"], device=DEV) // c["rows"]
            out["dgate"] = torch.zeros(st["gate"].shape, device=DEV).index_add_(0, at, p)
    return out


def _step_bwd_own(st):
    import expert_load_balance_amd as moe

    c, x = st["case"], st["x"]
    shape, H = _step_shape(moe, c), c["H"]
    out = {"dx": torch.empty_like(x), "dresidual": torch.empty_like(x), "dw_post": torch.empty(H, device=DEV),
           "dw_pre": torch.empty(H, device=DEV)}
    if st["gate"] is not None:
        out["dgate"] = torch.empty(st["gate"].shape, device=DEV)
    if "ws" not in st:  # kept from step to step
        st["ws"] = torch.empty(moe.moe_block_norm_backward_workspace_bytes(shape, _gate_rows(c)), dtype=torch.uint8, device=DEV)
    moe.moe_block_norm_backward(shape, x, st["rstd_post"], st["dy"], st["ds"], out["dx"], st["ws"], s=st["s"],
                                rstd_pre=st["rstd_pre"], alpha=st["alpha"], w_post=st["w_post"], gate=st["gate"],
                                gate_rows=_gate_rows(c), w_pre=st["w_pre"], dresidual=out["dresidual"],
                                dw_post=out["dw_post"], dgate=out.get("dgate"), dw_pre=out["dw_pre"])
    return out


_RUN = {"quant4": (_quant4_plain, _quant4_own), "experts4": (_experts4_plain, _experts4_own),
        "few": (_few_plain, _few_own), "step": (_step_plain, _step_own), "step_bwd": (_step_bwd_plain, _step_bwd_own)}


# ------------------------------------------------------------------- floors --

_SIZE = {BF16: 2.0, MX8: 1 + 1 / BLOCK, MX4: 0.5 + 1 / BLOCK}  # bytes a weight


def work(case):
    c = dict(case)
    if c["op"] == "quant4":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 if c["dtype"] == BF16 else 4) + n // 2 + n // BLOCK + 2 * n, "flops": 4 * n}
    if c["op"] in ("experts4", "few"):
        T, H, E, k, F = c["T"], c["H"], c["E"], c["k"], c["F"]
        live = E * (1 - (1 - k / E) ** T)  # experts that some token chose, drawn evenly
        if c["op"] == "experts4":
            return {"bytes": int(live * 3 * F * H * _SIZE[MX4]) + T * (H + H // BLOCK + 8 * k + 2 * H),
                    "flops": T * k * 6 * F * H + T * k * H * 2}
        return {"bytes": int((live * F + c["shared_F"]) * 3 * H * _SIZE[c["weights"]]) + E * (2 * H + 4) + 4 * T * H,
                "flops": T * (6 * H * (k * F + c["shared_F"]) + 2 * H * (E + k))}
    T, H, b = c["T"], c["H"], 2 if c["dtype"] == BF16 else 4
    gates = 0 if c["gate"] == "none" else T if c["gate"] == "token" else -(-T // c["rows"]) * H
    if c["op"] == "step":
        n = T * H * b * 4 + (2 * H + gates) * b + 8 * T
        if c["mx"]:
            n += T * H + T * (H // BLOCK)
        return {"bytes": n, "flops": T * H * (14 if c["mx"] else 11)}
    return {"bytes": T * H * b * 6 + (2 * H + gates) * b + (2 * H + gates) * 4 + 8 * T, "flops": T * H * 22}


# ------------------------------------------------------- the same in float64 --

def exact(case, seed):
    st = prepare(case, seed)
    return _EXACT[case["op"]](st)


def _nearest(v, values):
    """float64 magnitudes to the nearest of the table's (ascending), ties to the even place."""
    t = torch.tensor(values, dtype=torch.float64, device=v.device)
    a = v.abs()
    hi = torch.searchsorted(t, a.contiguous()).clamp(max=len(values) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = t[hi] - a, a - t[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(t[pick], v)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_E4M3 = [m / 512 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119]


def _scales64(top, largest):
    e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / largest)).clamp(min=-127)
    e = torch.where(top > largest * torch.exp2(e), e + 1, e)  # log2 landed a hair low
    e = torch.where((e > -127) & (top <= largest * torch.exp2(e - 1)), e - 1, e)
    return torch.exp2(e)


def _quant4_exact(st):
    x = st["x"]
    out = {"values": torch.empty(x.shape, dtype=torch.float64, device=x.device),
           "scales": torch.empty((x.shape[0], x.shape[1] // BLOCK), dtype=torch.float64, device=x.device)}
    for part, v, s in zip(*(t.split(max(1, (1 << 26) // x.shape[1])) for t in (x, out["values"], out["scales"]))):
        b = part.double().reshape(part.shape[0], -1, BLOCK)
        s.copy_(_scales64(b.abs().amax(-1), 6.0))
        v.copy_((_nearest(b / s[..., None], _E2M1) * s[..., None]).reshape(part.shape))
    return out


def _spread64(s, row):
    return s.double().repeat_interleave(BLOCK, dim=-1).reshape(row)


def _whole64(w, e):
    """float64 values of expert e of a projection in any form."""
    q, s = w[0][e], None if w[1] is None else w[1].view(torch.uint8)[e].view(w[1].dtype)
    if s is None:
        return q.double()
    if q.dtype == torch.uint8:
        t = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=q.device)
        both = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
        both[:, 0::2], both[:, 1::2] = t[(q % 16).int()], t[(q // 16).int()]
        return both * _spread64(s, both.shape)
    return q.double() * _spread64(s, q.shape)


def _swish64(g):
    return g / (1 + torch.exp(-g))


def _experts4_exact(st):
    c = st["case"]
    x = st["xq"].double() * _spread64(st["xs"], st["xq"].shape)
    w, ids = st["w"].double(), st["ids"].long()
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
    for e in st["live"].tolist():
        tok, j = (ids == e).nonzero(as_tuple=True)
        a = x[tok]
        h = _swish64(a @ _whole64(st["gate"], e).t()) * (a @ _whole64(st["up"], e).t())
        b = h.reshape(h.shape[0], -1, BLOCK)
        s = _scales64(b.abs().amax(-1), 448.0)[..., None]
        h = (_nearest(b / s, _E4M3) * s).reshape(h.shape)
        out.index_add_(0, tok, (h @ _whole64(st["down"], e).t()) * w[tok, j][:, None])
    return {"out": out}


def _few_exact(st):
    c = st["case"]
    x = st["x"].double()
    logits = x @ st["router"].double().t()
    # the score is one float32 addition; ties go to the lower expert
    order = torch.argsort(-(logits.float() + st["bias"]), dim=-1, stable=True)[:, :c["k"]]
    w = torch.softmax(logits.gather(1, order), -1)
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
    for e in order.unique().tolist():
        tok, j = (order == e).nonzero(as_tuple=True)
        a = x[tok]
        h = _swish64(a @ _whole64(st["gate"], e).t()) * (a @ _whole64(st["up"], e).t())
        out.index_add_(0, tok, (h @ _whole64(st["down"], e).t()) * w[tok, j][:, None])
    if st["shared"] is not None:
        g, u, d = (_whole64(m, 0) for m in st["shared"])
        out += (_swish64(x @ g.t()) * (x @ u.t())) @ d.t()
    return {"out": out}


def _gate64(st):
    c = st["case"]
    if st["gate"] is None:
        return torch.ones((), dtype=torch.float64, device=DEV)
    at = torch.arange(c["T"], device=DEV)
    return st["gate"].double()[at][:, None] if c["gate"] == "token" else st["gate"].double()[torch.div(at, c["rows"], rounding_mode="floor")]


def _step_exact(st):
    c, t = st["case"], _TYPES[st["case"]["dtype"]]
    x, H = st["x"].double(), st["case"]["H"]
    r1 = (x.pow(2).sum(-1) / H + EPS).pow(-0.5)
    s = st["alpha"] * st["residual"].double() + _gate64(st) * (x * r1[:, None] * st["w_post"].double())
    s = s.to(t).double()  # stored, and normed, in its type
    r2 = (s.pow(2).sum(-1) / H + EPS).pow(-0.5)
    y = s * r2[:, None] * st["w_pre"].double()
    out = {"s": s, "y": y, "rstd_post": r1, "rstd_pre": r2}
    if c["mx"]:
        b = y.reshape(c["T"], -1, BLOCK)
        out["scales"] = _scales64(b.abs().amax(-1), 448.0)
        out["q"] = _nearest(b / out["scales"][..., None], _E4M3).reshape(y.shape)
    return out


def _step_bwd_exact(st):
    c, H = st["case"], st["case"]["H"]
    x, s, dy, ds, w1, w2, r1, r2 = (st[n].double() for n in ("x", "s", "dy", "ds", "w_post", "w_pre", "rstd_post", "rstd_pre"))
    d = ds + dy * w2 * r2[:, None] - s * (r2.pow(3) * (dy * w2 * s).sum(-1) / H)[:, None]
    dn = d * _gate64(st)
    dx = dn * w1 * r1[:, None] - x * (r1.pow(3) * (dn * w1 * x).sum(-1) / H)[:, None]
    out = {"dx": dx, "dresidual": st["alpha"] * d, "dw_post": (dn * x * r1[:, None]).sum(0),
           "dw_pre": (dy * s * r2[:, None]).sum(0)}
    if st["gate"] is not None:
        n = d * x * r1[:, None] * w1
        if c["gate"] == "token":
            out["dgate"] = n.sum(-1)
        else:
            groups = torch.zeros((-(-c["T"] // c["rows"]) * c["rows"], H), dtype=torch.float64, device=DEV)
            groups[:c["T"]] = n
            out["dgate"] = groups.view(-1, c["rows"], H).sum(1)
    return out


_EXACT = {"quant4": _quant4_exact, "experts4": _experts4_exact, "few": _few_exact, "step": _step_exact,
          "step_bwd": _step_bwd_exact}
