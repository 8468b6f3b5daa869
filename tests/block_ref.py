"""Plain float64 forms of the operators around the layer, for the tests: the
formulas of include/moe_block.h, and bounds on how far a kernel that works in
float32 and rounds where the header says may be from them."""
import torch

U = 2.0 ** -24                                   # float32's half step
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def scale_byte(top):
    """e + 127 for block maxima (float64): the smallest e >= -127 with
    top <= 448 * 2^e; 255 where the block holds an infinity or NaN."""
    fin = torch.where(torch.isfinite(top), top, torch.ones_like(top))
    e = torch.arange(-127, 128, dtype=torch.float64, device=top.device)
    # first e that holds: the table's limits are exact in float64
    byte = torch.searchsorted(448.0 * torch.exp2(e), fin.contiguous())
    return torch.where(torch.isfinite(top), byte, torch.full_like(byte, 255))


def e4m3(v):
    """Nearest e4m3 value, ties to even, of float64 values up to 448."""
    _, x = torch.frexp(v)
    q = torch.exp2((x.double() - 1).clamp(min=-6) - 3)
    return torch.round(v / q) * q


def blocks(v, byte=None):
    """(dequantised float64 values, scale bytes) of rows cut into blocks of 32."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    if byte is None:
        a = b.abs()
        byte = scale_byte(torch.where(torch.isnan(a), torch.full_like(a, torch.inf), a).amax(-1))
    s = torch.exp2(byte.double() - 127)
    return (e4m3(b / s[..., None]) * s[..., None]).reshape(v.shape), byte


def values(q, s):
    """float64 values of codes and scale bytes."""
    f = q.view(torch.float8_e4m3fn).double()
    return f * torch.exp2(s.view(torch.uint8).double() - 127).repeat_interleave(32, -1)


def spread(v, d):
    """For exact values v known to +-d before they are cut into blocks: the
    dequantised form of v and how far another's may be from it."""
    ref, _ = blocks(v)
    b, t = v.reshape(*v.shape[:-1], -1, 32), d.reshape(*v.shape[:-1], -1, 32)
    lo = scale_byte((b.abs() - t).clamp(min=0).amax(-1))
    hi = scale_byte((b.abs() + t).amax(-1))
    far = torch.zeros_like(v)
    for byte in (lo, hi):
        for side in (-1, 1):
            far = torch.maximum(far, (blocks(v + side * d, byte)[0] - ref).abs())
    return ref, far


def check_blocks(q, s, v, d, what):
    """Codes and scale bytes against exact values v known to +-d."""
    b, t = v.reshape(*v.shape[:-1], -1, 32), d.reshape(*v.shape[:-1], -1, 32)
    s = s.view(torch.uint8).long()
    lo = scale_byte((b.abs() - t).clamp(min=0).amax(-1))
    hi = scale_byte((b.abs() + t).amax(-1))
    assert bool(((s >= lo) & (s <= hi)).all()), f"{what}: scale bytes"
    got = values(q, s.to(torch.uint8)).reshape(b.shape)
    unit = torch.exp2(s.double() - 127)[..., None]
    # half a step: 2^-4 of a normal value, 2^-10 of the scale below those
    tol = torch.maximum(b.abs() * 2.0 ** -4, unit * 2.0 ** -10) + t
    bad = ~((got - b).abs() <= tol * (1 + 1e-12))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} codes further than half a step"


def norm(x, residual, w, eps):
    """s (in x's type), rstd, v in float64."""
    s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    d = s.double()
    rstd = 1 / torch.sqrt(d.pow(2).mean(-1) + eps)
    return s, rstd, d * rstd[:, None] * w.double()


def norm_rel(H):
    """Relative error of rstd and of v where the squares are added in float32 (the
    kernel adds them in fp64, far within this): a thread adds up to
    max(4 * 8, H / 1024) squares in turn, then 6 steps of a wave and 16 waves;
    all terms are positive, so each add is off by U of a partial sum that is
    no more than the whole. The mean's error halves in the root; division,
    root, and two products round once each."""
    chain = max(32, H // 1024 + 8) + 6 + 16
    return (chain / 2 + 6) * U


def norm_bwd(s, w, rstd, dy, ds):
    """(dx, its bound before rounding, dweight, sum of |dy xhat|) in float64."""
    a, r, d, g = s.double(), rstd.double()[:, None], dy.double(), dy.double() * w.double()
    xh = a * r
    m, ma = (g * xh).mean(-1, keepdim=True), (g * xh).abs().mean(-1, keepdim=True)
    dx = r * (g - xh * m)
    H = s.shape[-1]
    chain = max(32, H // 1024 + 8) + 6 + 16 + 4
    tol = r * xh.abs() * (ma * chain * U) + 4 * U * (r * (g.abs() + (xh * m).abs()))
    if ds is not None:
        dx = dx + ds.double()
        tol = tol + 2 * U * ds.double().abs()
    return dx, tol, (d * xh).sum(0), (d * xh).abs().sum(0)


def _codes(v, byte):
    """(magnitudes, exponents) of the codes of dequantised rows, and their
    blocks' scales; the exponent of a subnormal code is that of its format, -6."""
    c = (v.reshape(*v.shape[:-1], -1, 32) / torch.exp2(byte.double() - 127)[..., None]).reshape(v.shape).float().abs()
    _, x = torch.frexp(c)
    return c, (x - 1).clamp(min=-6), torch.exp2(byte.float() - 127)


def truncation(x, xb, w, wb):
    """Most that the matrix instruction drops from x @ w.T (dequantised rows
    and their scale bytes). It adds the products of 8 neighbouring codes as
    integers: each product, of exponent ex + ew and 6 fraction bits, is cut
    toward zero to a multiple of 2^(m - 13), m the largest exponent sum of the
    eight (measured on the instruction: beside 2^16, 2.25 * 2^4 counts as 32 and
    2^2 as nothing). So a product loses something only where its exponent is
    below m - 7, and then less than 2^(m - 13) and no more than itself."""
    cx, ex, sx = _codes(x, xb)
    cw, ew, sw = _codes(w, wb)
    out = torch.zeros((x.shape[0], w.shape[0]), device=x.device)
    for k in range(0, x.shape[1], 8):
        e = ex[:, None, k:k + 8] + ew[None, :, k:k + 8]
        p = cx[:, None, k:k + 8] * cw[None, :, k:k + 8]
        m = torch.where(p > 0, e, torch.full_like(e, -99)).amax(-1, keepdim=True)
        lost = torch.where(e < m - 7, torch.minimum(p, torch.exp2((m - 13).float())), torch.zeros_like(p)).sum(-1)
        out += lost * sx[:, None, k // 32] * sw[None, :, k // 32]
    return out.double()


def experts(a, a_bytes, e_of, wg, wu, wd):
    """y (float64) and its bound before bf16's rounding for rows `a` (float64
    values with their scale bytes) of experts e_of; weights as (codes, bytes)."""
    y = torch.zeros((a.shape[0], wd[0].shape[1]), dtype=torch.float64, device=a.device)
    tol = torch.zeros_like(y)
    H, F = wg[0].shape[2], wg[0].shape[1]
    # what the eights leave is added in float32, 64 products to an instruction:
    # each of the K / 64 adds is off by at most 2^-22 of the magnitudes added;
    # the sums of up to 32 K-parts round 32 times more
    cH, cF = (H / 64 + 32) * 2.0 ** -22, (F / 64 + 32) * 2.0 ** -22
    for e in torch.unique(e_of).tolist():
        rows = (e_of == e).nonzero().reshape(-1)
        G, Up, D = values(wg[0][e], wg[1][e]), values(wu[0][e], wu[1][e]), values(wd[0][e], wd[1][e])
        for r in rows.split(512):
            x, xb = a[r], a_bytes[r]
            g, u = x @ G.t(), x @ Up.t()
            dg = truncation(x, xb, G, wg[1][e]) + cH * (x.abs() @ G.abs().t())
            du = truncation(x, xb, Up, wu[1][e]) + cH * (x.abs() @ Up.abs().t())
            silu = g * torch.sigmoid(g)
            # exp2 and reciprocal are good to 1 ulp each; z log2(e) carries 2^-24
            # of z into the exponent; |silu'| <= 1.1
            h = silu * u
            dh = (h.abs() * (g.abs() * 1.5 + 8) * 2.0 ** -23 + 1.1 * dg * u.abs() + silu.abs() * du
                  + 1.1 * dg * du)
            hq, far = spread(h, dh)
            y[r] = hq @ D.t()
            # a code of h that is a step off can double what its eight drops
            drop = 2 * truncation(hq, blocks(h)[1], D, wd[1][e])
            tol[r] = far @ D.abs().t() + drop + cF * ((hq.abs() + far) @ D.abs().t())
    return y, tol
