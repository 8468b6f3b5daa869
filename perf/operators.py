"""The operators around one MoE layer: what is computed, on which sizes, and
their plain forms.

Four operators:

  norm      root-mean-square norm of the residual stream with the residual's
            addition, its result in the activation type and, for the experts'
            8-bit products, in e4m3 with one power-of-two scale per 32 columns;
  norm_bwd  its backward: the gradient of the residual stream and of the norm's
            weight;
  experts   the routed experts' SwiGLU block on 8-bit rows and 8-bit weights
            (dispatch, both products, gate-weighted combine);
  clip      the global norm over a list of gradients, and the gradients clipped
            to it.

``own`` False computes them with elementary torch operations in float32; True
calls the library. ``exact`` computes them in float64.

8-bit blocks: 32 consecutive values of a row share the scale 2^e, e the
smallest integer >= -127 with max|v| <= 448 * 2^e (448 is e4m3's largest
value, so nothing saturates); the values are v / 2^e rounded to nearest even.
The scale is stored as the byte e + 127. Codes and scales are handed over as
torch's float8_e4m3fn and float8_e8m0fnu tensors, whose elements are the values
that the bytes stand for.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}
BLOCK = 32


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one token of a decode step in front of a layer 4096 wide: latency
        dict(name="norm_decode_1", op="norm", T=1, H=4096, dtype=BF16, residual=True, mx=True),
        # a prefill batch 7168 wide: residual added, both outputs
        dict(name="norm_prefill_8192", op="norm", T=8192, H=7168, dtype=BF16, residual=True, mx=True),
        # a float32 model's first norm (no residual yet), odd token count and width
        dict(name="norm_f32_1021", op="norm", T=1021, H=2052, dtype=F32, residual=False, mx=False),
        # training, the widest batch: gradient through the norm and past it
        dict(name="norm_bwd_8192", op="norm_bwd", T=8192, H=7168, dtype=BF16, residual=True),
        # training a small float32 model: few rows, odd sizes, no second gradient
        dict(name="norm_bwd_f32_333", op="norm_bwd", T=333, H=1540, dtype=F32, residual=False),
        # decoding one token: 8 of 128 experts, each with one row
        dict(name="experts_decode_1", op="experts", T=1, H=4096, E=128, k=8, F=1536, R=16, skew=0.0),
        # a decode batch: every expert with a few rows, some with many
        dict(name="experts_decode_256", op="experts", T=256, H=4096, E=128, k=8, F=1536, R=16, skew=0.2),
        # a prefill chunk over many narrow experts
        dict(name="experts_a3b_4096", op="experts", T=4096, H=2048, E=128, k=8, F=768, R=16, skew=0.2),
        # few wide experts, a ragged token count: bound by the matrix cores
        dict(name="experts_mixtral_2047", op="experts", T=2047, H=4096, E=8, k=2, F=14336, R=8, skew=0.1),
        # the largest layer: 11 GB of expert weights against 65536 rows
        dict(name="experts_dsv3_8192", op="experts", T=8192, H=7168, E=256, k=8, F=2048, R=32, skew=0.2),
        # norms, routers and small dense weights of a deep model: 96 tensors,
        # bfloat16 beside float32, few bytes: launches and lookups count
        dict(name="clip_many_small", op="clip", layers=24, H=2048, E=128, F=768, experts=False, dtype=BF16),
        # one layer's expert gradients in float32, 5.6 GB
        dict(name="clip_experts_f32", op="clip", layers=1, H=4096, E=8, F=14336, experts=True, dtype=F32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "experts", "experts", "clip"])
    if op in ("norm", "norm_bwd"):
        dtype = rng.choice([BF16, BF16, F32])
        T = _log(rng, 1, 8192)
        c = dict(op=op, T=T, dtype=dtype, residual=rng.random() < 0.7)
        mx = op == "norm" and rng.random() < 0.6
        step = 64 if dtype == BF16 else 32 if mx else 4
        c["H"] = max(1, _log(rng, 64, 8192) // step) * step
        while c["T"] * c["H"] > 8192 * 7168 // (1 if dtype == BF16 else 2):
            c["T"] = c["T"] // 2 + 1
        if op == "norm":
            c["mx"] = mx
        return c
    if op == "experts":
        while True:
            E = rng.choice([4, 6, 8, 16, 40, 64, 96, 128, 256])
            R = rng.choice([r for r in range(1, 33) if E % r == 0])
            k = rng.randint(1, min(8, E))
            H = _log(rng, 128, 7168) // 128 * 128
            F = _log(rng, 128, 8192) // 128 * 128
            T = _log(rng, 1, 8192)
            if E * 3 * F * H <= 4 << 30 and T * k * 6 * F * H <= 4e12:
                return dict(op=op, T=T, H=H, E=E, k=k, F=F, R=R, skew=round(rng.uniform(0, 0.6), 2))
    while True:
        H, F, E = _log(rng, 64, 7168), _log(rng, 32, 8192), rng.choice([4, 8, 16, 64, 128])
        c = dict(op="clip", layers=_log(rng, 1, 48), H=H, E=E, F=F, experts=rng.random() < 0.5,
                 dtype=rng.choice([BF16, F32]))
        if sum(math.prod(s) for s, _ in _clip_shapes(c)) <= 1_000_000_000:
            return c


def _clip_shapes(c):
    """(shape, float32) of every gradient: per layer the norm's weight (float32),
    the router's, and the weights of a shared expert or of all experts (F x H)."""
    out = []
    wide = c["dtype"] == F32
    for _ in range(c["layers"]):
        out.append(((c["H"],), True))
        out.append(((c["E"], c["H"]), wide))
        e = c["E"] if c["experts"] else 1
        out.append(((e, c["F"], c["H"]), wide))
        if c["experts"]:
            out.append(((e, c["F"], c["H"]), wide))
        out.append(((e, c["H"], c["F"]), wide))
    return out


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1_000_003 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _channels(g, H):
    """Per-channel spread of a residual stream: most near 1, a few 10 and more."""
    return torch.exp(_randn(g, H) * 0.5) * (1 + 15 * (torch.rand(H, generator=g, device=DEV) < 0.004))


def _pack(v):
    """(e4m3 codes, e8m0 scales) of float32 rows, 32 columns to a scale."""
    b = v.view(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)
    top = b.abs().amax(-1)
    m, x = torch.frexp(top)
    e = x - 9 + (m > 0.875).to(torch.int32)
    e = torch.where(top == 0, torch.full_like(e, -127), e.clamp(min=-127))
    q = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(v.shape), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _weights(g, E, rows, cols):
    q = torch.empty((E, rows, cols), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty((E, rows, cols // BLOCK), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (rows * cols))
    for a in range(0, E, step):
        b = min(E, a + step)
        qa, sa = _pack(_randn(g, b - a, rows, cols) / math.sqrt(cols))
        q[a:b].view(torch.uint8).copy_(qa.view(torch.uint8))
        s[a:b].copy_(sa.view(torch.uint8))
    return q, s.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    st = {"case": c}
    if c["op"] in ("norm", "norm_bwd"):
        T, H, t = c["T"], c["H"], _TYPES[c["dtype"]]
        ch = _channels(g, H)
        st["x"] = (_randn(g, T, H) * ch).to(t)
        st["weight"] = (1 + 0.2 * _randn(g, H)).to(t)
        if c["op"] == "norm":
            st["residual"] = (_randn(g, T, H) * ch).to(t) if c["residual"] else None
        else:
            st["dy"] = _randn(g, T, H).to(t)
            st["ds"] = _randn(g, T, H).to(t) if c["residual"] else None
            # what the forward kept
            st["rstd"] = torch.rsqrt(st["x"].double().square().mean(-1) + EPS).float()
    elif c["op"] == "experts":
        T, H, E, k, F = c["T"], c["H"], c["E"], c["k"], c["F"]
        x = _randn(g, T, H) * _channels(g, H)
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True))
        st["xq"], st["xs"] = _pack(x)
        rank = torch.randperm(E, generator=g, device=DEV).float()
        logits = _randn(g, T, E)
        ids = torch.topk(logits - c["skew"] * torch.log1p(rank), k, dim=-1).indices
        st["w"] = torch.softmax(torch.gather(logits, 1, ids), -1)
        st["ids"] = ids.to(torch.int32)
        st["gate"] = _weights(g, E, F, H)
        st["up"] = _weights(g, E, F, H)
        st["down"] = _weights(g, E, H, F)
        # the plain form's padding: experts with rows, and the most rows of one
        counts = torch.bincount(ids.reshape(-1), minlength=E)
        st["live"] = counts.nonzero().reshape(-1)
        st["most"] = int(counts.max())
    else:
        shapes = _clip_shapes(c)
        n32 = sum(math.prod(s) for s, wide in shapes if wide)
        n16 = sum(math.prod(s) for s, wide in shapes if not wide)
        st["flat"] = {"f32": torch.empty(n32, device=DEV), "bf16": torch.empty(n16, dtype=torch.bfloat16, device=DEV)}
        st["into"] = {n: torch.empty_like(v) for n, v in st["flat"].items()}
        at = {"f32": 0, "bf16": 0}
        st["grads"], st["clipped"] = [], []
        for i, (shape, wide) in enumerate(shapes):
            name, n = "f32" if wide else "bf16", math.prod(shape)
            v = st["flat"][name][at[name]:at[name] + n]
            for a in range(0, n, 1 << 28):
                b = min(n, a + (1 << 28))
                v[a:b] = _randn(g, b - a) * (10.0 ** (-(i % 4)))
            st["grads"].append(v.view(shape))
            st["clipped"].append(st["into"][name][at[name]:at[name] + n].view(shape))
            at[name] += n
        st["max_norm"] = 1.0
    return st


# --------------------------------------------------------------- one pass ----

def run(state):
    return _RUN[state["case"]["op"]][1 if own else 0](state)


def _norm_plain(st):
    c, t = st["case"], _TYPES[st["case"]["dtype"]]
    s = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(t)
    sf = s.float()
    rstd = torch.rsqrt(sf.square().mean(-1) + EPS)
    y = sf * rstd.unsqueeze(-1) * st["weight"].float()
    out = {"y": y.to(t), "rstd": rstd}
    if st["residual"] is not None:
        out["s"] = s
    if c["mx"]:
        out["q"], out["scales"] = _pack(y)
    return out


def _norm_own(st):
    import expert_load_balance_amd as moe

    c, x = st["case"], st["x"]
    T, H = c["T"], c["H"]
    shape = moe.Shape(T, H, 1, 1, 64, 1, 0, moe.MOE_BF16 if c["dtype"] == BF16 else moe.MOE_F32)
    out = {"y": torch.empty_like(x), "rstd": torch.empty(T, device=x.device)}
    if st["residual"] is not None:
        out["s"] = torch.empty_like(x)
    if c["mx"]:
        out["q"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=x.device)
        out["scales"] = torch.empty((T, H // BLOCK), dtype=torch.float8_e8m0fnu, device=x.device)
    moe.moe_rmsnorm(shape, x, st["weight"], EPS, residual=st["residual"], s=out.get("s"), y=out["y"],
                    q=out.get("q"), scales=out.get("scales"), rstd=out["rstd"])
    return out


def _norm_bwd_plain(st):
    t = _TYPES[st["case"]["dtype"]]
    xhat = st["x"].float() * st["rstd"].unsqueeze(-1)
    dy = st["dy"].float()
    gw = dy * st["weight"].float()
    dx = (gw - xhat * (gw * xhat).mean(-1, keepdim=True)) * st["rstd"].unsqueeze(-1)
    if st["ds"] is not None:
        dx = dx + st["ds"].float()
    return {"dx": dx.to(t), "dweight": (dy * xhat).sum(0)}


def _norm_bwd_own(st):
    import expert_load_balance_amd as moe

    c, x = st["case"], st["x"]
    T, H = c["T"], c["H"]
    shape = moe.Shape(T, H, 1, 1, 64, 1, 0, moe.MOE_BF16 if c["dtype"] == BF16 else moe.MOE_F32)
    out = {"dx": torch.empty_like(x), "dweight": torch.empty(H, device=x.device)}
    if "ws" not in st:  # kept from step to step
        st["ws"] = torch.empty(max(moe.moe_rmsnorm_backward_workspace_bytes(shape), 16),
                               dtype=torch.uint8, device=x.device)
    moe.moe_rmsnorm_backward(shape, x, st["weight"], st["rstd"], st["dy"], out["dx"], out["dweight"],
                             st["ws"], ds=st["ds"])
    return out


def _values(q, s):
    """float32 values of 8-bit blocks."""
    b = q.float().view(*s.shape, BLOCK)
    return (b * s.float().unsqueeze(-1)).view(q.shape)


def _bytes_at(t, i):
    """Rows i of an 8-bit tensor."""
    return t.view(torch.uint8)[i].view(t.dtype)


def _experts_plain(st):
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
    rows[slot, place] = _values(st["xq"], st["xs"])[order // k]

    def times(a, w):
        return torch.bmm(a, _values(_bytes_at(w[0], live), _bytes_at(w[1], live)).transpose(1, 2))

    g = times(rows, st["gate"])
    h = g * torch.sigmoid(g) * times(rows, st["up"])
    y = times(_values(*_pack(h)), st["down"])[slot, place]
    per = torch.empty((T * k, H), device=DEV)
    per[order] = y
    return {"out": (per.view(T, k, H) * st["w"].unsqueeze(-1)).sum(1).to(torch.bfloat16)}


def _experts_own(st):
    import expert_load_balance_amd as moe

    c = st["case"]
    T, H, k = c["T"], c["H"], c["k"]
    if "layer" not in st:  # buffers and workspace that a program keeps per shape
        from expert_load_balance_amd.layer import MoeLayerMx

        st["layer"] = MoeLayerMx(moe.Shape(T, H, c["E"], k, c["F"], c["R"], 0, moe.MOE_BF16), DEV)
    return {"out": st["layer"].experts(st["xq"], st["xs"], st["ids"], st["w"], st["gate"], st["up"], st["down"])}


def _clip_plain(st):
    total = torch.stack([g.double().square().sum() for g in st["grads"]]).sum().sqrt()
    scale = torch.where(total > st["max_norm"], st["max_norm"] / total, torch.ones_like(total))
    for g, o in zip(st["grads"], st["clipped"]):
        o.copy_((g.float() * scale.float()).to(o.dtype))
    return {"norm": total.float(), "f32": st["into"]["f32"], "bf16": st["into"]["bf16"]}


def _clip_own(st):
    import expert_load_balance_amd as moe

    if "ws" not in st:  # kept from step to step
        st["ws"] = torch.empty(moe.moe_grad_workspace_bytes(st["grads"]), dtype=torch.uint8, device=DEV)
        st["norm"] = torch.empty(1, device=DEV)
        st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_grad_norm(st["grads"], st["norm"], st["err"], st["ws"])
    moe.moe_grad_clip(st["grads"], st["clipped"], st["max_norm"], st["norm"])
    return {"norm": st["norm"].view(()), "f32": st["into"]["f32"], "bf16": st["into"]["bf16"]}


_RUN = {"norm": (_norm_plain, _norm_own), "norm_bwd": (_norm_bwd_plain, _norm_bwd_own),
        "experts": (_experts_plain, _experts_own), "clip": (_clip_plain, _clip_own)}


# ------------------------------------------------------------------- floors --

def work(case):
    c = dict(case)
    if c["op"] in ("norm", "norm_bwd"):
        T, H, b = c["T"], c["H"], 2 if c["dtype"] == BF16 else 4
        if c["op"] == "norm":
            n = T * H * b * (4 if c["residual"] else 2) + H * b + T * 4
            if c["mx"]:
                n += T * H + T * (H // BLOCK)
            return {"bytes": n, "flops": T * H * (8 if c["mx"] else 5)}
        return {"bytes": T * H * b * (4 if c["residual"] else 3) + H * (b + 4) + T * 4, "flops": T * H * 10}
    if c["op"] == "experts":
        T, H, E, k, F = c["T"], c["H"], c["E"], c["k"], c["F"]
        live = E * (1 - (1 - k / E) ** T)  # experts that some token chose, drawn evenly
        row = H + H // BLOCK
        return {"bytes": int(live * 3 * F * H * (1 + 1 / BLOCK)) + T * (row + 8 * k + 2 * H),
                "flops": T * k * 6 * F * H + T * k * H * 2}
    n = sum(math.prod(s) * (4 if wide else 2) for s, wide in _clip_shapes(c))
    m = sum(math.prod(s) for s, _ in _clip_shapes(c))
    return {"bytes": 2 * n + 4, "flops": 3 * m}


# ------------------------------------------------------- the same in float64 --

def _round_e4m3(v):
    """float64 values to the nearest e4m3 value, ties to even (|v| <= 448)."""
    _, x = torch.frexp(v.abs())
    quantum = torch.exp2((x.double() - 1).clamp(min=-6) - 3)
    return torch.round(v / quantum) * quantum


def _blocks64(v):
    """(rounded quotients, scales) of float64 rows."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    top = b.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448)).clamp(min=-127)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)  # log2 landed a hair low
    e = torch.where((e > -127) & (top <= 448 * torch.exp2(e - 1)), e - 1, e)
    s = torch.exp2(e)
    return _round_e4m3(b / s.unsqueeze(-1)).reshape(v.shape), s


def exact(case, seed):
    st = prepare(case, seed)
    return _EXACT[case["op"]](st)


def _norm_exact(st):
    t = _TYPES[st["case"]["dtype"]]
    s = st["x"].double()
    if st["residual"] is not None:
        s = (s + st["residual"].double()).to(t).double()  # the sum is stored, and normed, in its type
    rstd = (s.pow(2).sum(-1) / s.shape[-1] + EPS).pow(-0.5)
    y = s * rstd[:, None] * st["weight"].double()
    out = {"y": y, "rstd": rstd}
    if st["residual"] is not None:
        out["s"] = s
    if st["case"]["mx"]:
        out["q"], out["scales"] = _blocks64(y)
    return out


def _norm_bwd_exact(st):
    x, r, dy, w = (st[n].double() for n in ("x", "rstd", "dy", "weight"))
    H = x.shape[-1]
    dot = (dy * w * x).sum(-1)
    dx = dy * w * r[:, None] - x * (r.pow(3) * dot / H)[:, None]
    if st["ds"] is not None:
        dx = dx + st["ds"].double()
    return {"dx": dx, "dweight": (dy * (x * r[:, None])).sum(0)}


def _experts_exact(st):
    c = st["case"]
    T, H = c["T"], c["H"]

    def value(q, s):
        return q.double() * s.double().repeat_interleave(BLOCK, dim=-1)

    x = value(st["xq"], st["xs"])
    w = st["w"].double()
    ids = st["ids"].long()
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for e in st["live"].tolist():
        tok, j = (ids == e).nonzero(as_tuple=True)
        wg, wu, wd = (value(st[n][0][e], st[n][1][e]) for n in ("gate", "up", "down"))
        a = x[tok]
        g = a @ wg.t()
        q, s = _blocks64(g / (1 + torch.exp(-g)) * (a @ wu.t()))
        h = q * s.repeat_interleave(BLOCK, dim=-1)
        out.index_add_(0, tok, (h @ wd.t()) * w[tok, j][:, None])
    return {"out": out}


def _clip_exact(st):
    sq = torch.zeros((), dtype=torch.float64, device=DEV)
    for g in st["grads"]:
        f = g.reshape(-1)
        for a in range(0, f.numel(), 1 << 27):
            sq += f[a:a + (1 << 27)].double().pow(2).sum()
    norm = sq.sqrt()
    c = (st["max_norm"] / norm).clamp(max=1.0)
    return {"norm": norm, "f32": st["flat"]["f32"].double() * c, "bf16": st["flat"]["bf16"].double() * c}


_EXACT = {"norm": _norm_exact, "norm_bwd": _norm_bwd_exact, "experts": _experts_exact, "clip": _clip_exact}
