"""Plain float64 forms of the operators of include/moe_step.h, for the tests, and
bounds on how far a kernel that works in float32 and rounds where the header says
may be from them. U is float32's half step; block_ref.HALF a type's."""
import torch

from block_ref import HALF, U, scale_byte as scale_byte8  # noqa: F401

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------- 4-bit blocks ----

def scale_byte4(top):
    """e + 127 for block maxima (float64): the smallest e >= -127 with top <= 6 *
    2^e; 255 where the block holds an infinity or NaN."""
    fin = torch.where(torch.isfinite(top), top, torch.ones_like(top))
    e = torch.arange(-127, 128, dtype=torch.float64, device=top.device)
    byte = torch.searchsorted(6.0 * torch.exp2(e), fin.contiguous())
    return torch.where(torch.isfinite(top), byte, torch.full_like(byte, 255))


def codes4(v):
    """(codes 0..15 of every value, scale bytes) of float64 rows: the nearest of
    the eight magnitudes, a tie to the one with the even code."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    a = b.abs()
    byte = scale_byte4(torch.where(torch.isnan(a), torch.full_like(a, torch.inf), a).amax(-1))
    r = a / torch.exp2(byte.double() - 127)[..., None]
    t = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    far = (r[..., None] - t).abs()
    # (the even code of a tie: order the table by code % 2, then take the first minimum)
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=v.device)
    code = order[far[..., order].argmin(-1)] + 8 * torch.signbit(b)
    code = torch.where((byte == 255)[..., None], torch.zeros_like(code), code)
    return code.reshape(v.shape).to(torch.uint8), byte.to(torch.uint8)


def pack4(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack4(q):
    q = q.view(torch.uint8)
    return torch.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], 2 * q.shape[-1])


def values4(q, s):
    """float64 values of packed codes and scale bytes (NaN where the byte is 255)."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=q.device)
    byte = s.view(torch.uint8)
    f = torch.where(byte == 255, torch.full(byte.shape, torch.nan, dtype=torch.float64, device=q.device),
                    torch.exp2(byte.double() - 127))
    return t[unpack4(q).long()] * f.repeat_interleave(32, -1)


# --------------------------------------------------- norms between two blocks ----

def gate_rows_of(gate, rows, T):
    """The gate as it multiplies the rows, float64."""
    if gate is None:
        return torch.ones((), dtype=torch.float64)
    g = gate.double()
    return g[:, None] if rows == 0 else g.repeat_interleave(rows, 0)[:T]


def rstd(x, eps):
    return 1 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)


def block_norm(x, residual, alpha, w_post, gate, rows, w_pre, eps):
    """s before its rounding, its bound, rstd_post. The mean is a sum in fp64, so
    rstd is off by one rounding; n takes two products, the gate one, the addition
    one and alpha's product may be one more: at most 6 roundings of either term."""
    x = x.double()
    r1 = rstd(x, eps)
    n = x if w_post is None else x * r1 * w_post.double()
    a = gate_rows_of(gate, rows, x.shape[0]).to(x.device) * n
    b = torch.zeros_like(a) if residual is None else alpha * residual.double()
    return a + b, 6 * U * (a.abs() + b.abs()), r1[:, 0]


def pre_norm(s, w_pre, eps):
    """(v, its bound, rstd_pre) from the stored s: rstd and two products round."""
    s = s.double()
    r2 = rstd(s, eps)
    v = s * r2 * w_pre.double()
    return v, 4 * U * v.abs(), r2[:, 0]


def chain(H):
    """Adds in turn on the way of a float32 sum over a row: a thread's own, a wave's
    six steps, sixteen waves."""
    return max(32, H // 1024 + 8) + 6 + 16 + 4


def block_norm_bwd(x, r1, s, r2, alpha, w_post, gate, rows, w_pre, dy, ds):
    """{output: (value, bound before rounding)}. Each of the formula's products and
    sums rounds once; C counts those of any one term generously (10)."""
    C, T, H = 10 * U, x.shape[0], x.shape[1]
    x = x.double()
    zero = torch.zeros_like(x)
    d, td = (zero, zero) if ds is None else (ds.double(), 2 * U * ds.double().abs())
    out = {}
    if dy is not None:
        r, dyd = r2.double()[:, None], dy.double()
        sh, g = s.double() * r, dyd * w_pre.double()
        m, ma = (g * sh).mean(-1, keepdim=True), (g * sh).abs().mean(-1, keepdim=True)
        d = d + r * (g - sh * m)
        td = td + r * sh.abs() * ma * chain(H) * U + C * r * (g.abs() + sh.abs() * ma)
        out["dw_pre"] = ((dyd * sh).sum(0), (T + 44) * U * (dyd * sh).abs().sum(0))
    out["dresidual"] = (alpha * d, abs(alpha) * (td + U * d.abs()))
    r = r1.double()[:, None] if w_post is not None else torch.ones_like(x[:, :1])
    xh = x * r
    n = xh if w_post is None else xh * w_post.double()
    g = gate_rows_of(gate, rows, T).to(x.device)
    if gate is not None:
        p, tp = d * n, td * n.abs() + C * (d * n).abs()
        if rows == 0:  # (two sums, as for dx below)
            big = zero if ds is None else ds.double().abs()
            if dy is not None:
                big = big + r2.double()[:, None] * (dyd * w_pre.double()).abs() + r2.double()[:, None] * sh.abs() * ma
            out["dgate"] = (p.sum(-1), tp.sum(-1) + (chain(H) * U + C) * (n.abs() * big).sum(-1))
        else:
            at = torch.arange(T, device=x.device) // rows
            k = gate.shape[0]

            def groups(v):
                return torch.zeros((k, H), dtype=torch.float64, device=x.device).index_add_(0, at, v)

            out["dgate"] = (groups(p), groups(tp) + (min(rows, T) + 44) * U * groups(p.abs()))
    dn = g * d
    tdn = g.abs() * (td + C * d.abs())
    if w_post is None:
        out["dx"] = (dn, tdn)
        return out
    w = w_post.double()
    e, te = dn * w, tdn * w.abs()
    m = (e * xh).mean(-1, keepdim=True)
    # the mean is a difference of two sums, of what ds and dy give and of what the
    # first mean takes away: their terms' magnitudes count, not those of d
    big = (g * w * xh).abs()
    parts = zero if ds is None else ds.double().abs()
    if dy is not None:
        parts = parts + r2.double()[:, None] * (dyd * w_pre.double()).abs() + r2.double()[:, None] * sh.abs() * ma
    tm = (te * xh.abs()).mean(-1, keepdim=True) + (chain(H) * U + C) * (big * parts).mean(-1, keepdim=True)
    out["dx"] = (r * (e - xh * m), r * (te + xh.abs() * tm) + C * r * (e.abs() + (xh * m).abs()))
    out["dw_post"] = ((dn * xh).sum(0), (tdn * xh.abs() + C * (dn * xh).abs()).sum(0) + (T + 44) * U * (dn * xh).abs().sum(0))
    return out


def check(got, want, what, t=None):
    """got within the bound, and half a step of its type where it is rounded."""
    v, tol = want
    if t is not None:
        tol = HALF[t] * (v.abs() + tol) + tol + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    off = (got.double() - v).abs()
    bad = ~(off <= tol * (1 + 1e-9) + 1e-300)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} out, worst {float((off / tol.clamp(min=1e-300)).max()):.3f} of its bound"


# ----------------------------------------------------- the layer for a few tokens ----

def whole(w, e):
    """float64 values of expert e of (values, scales)."""
    v, s = w
    if s is None:
        return v[e].double()
    if v.dtype == torch.uint8 and v.shape[-1] * 2 == s.shape[-1] * 32:
        return values4(v[e], s[e])
    return v[e].view(torch.float8_e4m3fn).double() * torch.exp2(s[e].view(torch.uint8).double() - 127).repeat_interleave(32, -1)


def swiglu(x, gate, up, down):
    """y and its bound for float64 rows x and one expert's float64 weights, products
    of bf16 values with fp32 sums. A matrix instruction adds 32 products to its sum,
    off by at most 2^-22 of the magnitudes added; eight waves share K and add up at
    the end. h is two bf16: 2^-17 of it is lost at most. exp and the quotient are
    good to 2 ulp, |silu'| <= 1.1."""
    H, F = gate.shape[1], gate.shape[0]
    cH, cF = (H / 256 + 12) * 2.0 ** -22, (F / 128 + 24) * 2.0 ** -22
    g, u = x @ gate.t(), x @ up.t()
    dg, du = cH * (x.abs() @ gate.abs().t()), cH * (x.abs() @ up.abs().t())
    silu = g * torch.sigmoid(g)
    h = silu * u
    dh = h.abs() * ((g.abs() * 1.5 + 8) * 2.0 ** -23 + 2.0 ** -17) + 1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du
    return h @ down.t(), dh @ down.abs().t() + cF * ((h.abs() + dh) @ down.abs().t())


def logits_of(x, wr):
    """Router scores and their bound: a wave adds up to four matrix instructions of 32
    products (each off by at most 2^-22 = 4 U of the magnitudes added), then eight
    waves and up to eight parts of H are added: 16 + 8 + 8 roundings of U."""
    z, a = x.double() @ wr.double().t(), x.double().abs() @ wr.double().abs().t()
    return z, 32 * U * a


def few(x, wr, bias, ids, gate, up, down, shared=None):
    """(out, its bound before rounding, w, its bound) for the choice `ids`, and
    whether ids is a top-k of logits + bias as far as float32 can tell."""
    z, dz = logits_of(x, wr)
    score = z if bias is None else z + bias.double()
    ds = dz + U * score.abs()
    ids = ids.long()
    taken = torch.zeros_like(z, dtype=torch.bool).scatter_(1, ids, True)
    assert bool((taken.sum(-1) == ids.shape[1]).all()), "an expert twice"
    low = torch.where(taken, score + ds, torch.full_like(score, torch.inf)).amin(-1)
    high = torch.where(taken, torch.full_like(score, -torch.inf), score - ds).amax(-1)
    fine = bool((low >= high).all())
    s, d = score.gather(1, ids), ds.gather(1, ids)
    fine = fine and bool((s[:, :-1] + d[:, :-1] >= s[:, 1:] - d[:, 1:]).all())
    l, dl = z.gather(1, ids), dz.gather(1, ids)
    w = torch.softmax(l, -1)
    dw = w * (2 * dl.amax(-1, keepdim=True) + 2 * (l - l.amax(-1, keepdim=True)).abs() * 2.0 ** -23 + 12 * U)
    T, k = ids.shape
    out = torch.zeros((T, down[0].shape[1]), dtype=torch.float64, device=x.device)
    tol, mag = torch.zeros_like(out), torch.zeros_like(out)
    xd = x.double()
    for e in torch.unique(ids).tolist():
        tok, j = (ids == e).nonzero(as_tuple=True)
        y, dy = swiglu(xd[tok], whole(gate, e), whole(up, e), whole(down, e))
        a, b = w[tok, j][:, None], dw[tok, j][:, None]
        out.index_add_(0, tok, a * y)
        tol.index_add_(0, tok, a * dy + b * (y.abs() + dy))
        mag.index_add_(0, tok, a * y.abs())
    if shared is not None:
        y, dy = swiglu(xd, *(whole(m, 0) for m in shared))
        out, tol, mag = out + y, tol + dy, mag + y.abs()
    return out, tol + (k + 6) * U * (mag + tol), w, dw, fine
