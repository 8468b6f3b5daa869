"""The operators of include/moe_step.h in a row, as a model calls them: serving steps
(norms between two blocks, router, experts on 4-bit weights or the layer for a few
tokens, the next norms), eager and from a graph, and the gradient of a stack of
blocks through the norms between them."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402
from expert_load_balance_amd.layer import MoeLayerFew, MoeLayerMx  # noqa: E402

import step_ref as ref  # noqa: E402
from test_gpu_experts4 import check as check_experts  # noqa: E402
from test_gpu_few import BF, DEV, blocks, check as check_few, gen, randn  # noqa: E402

pytestmark = pytest.mark.gpu
EPS, ALPHA = 1e-5, 0.75


class Step:
    """x (a block's output) and the stream it read -> norms -> MoE layer -> norms."""

    def __init__(self, T, H, E, k, F, few, seed):
        g = gen(seed)
        self.shape = moe.Shape(T, H, E, k, F, 2, 1, moe.MOE_BF16)
        self.x, self.r = randn(g, T, H).to(BF), randn(g, T, H).to(BF)
        self.w_post, self.w_pre, self.w_last = (1 + 0.2 * randn(g, H) for _ in range(3))
        self.w_post, self.w_pre, self.w_last = (w.to(BF) for w in (self.w_post, self.w_pre, self.w_last))
        self.gate = torch.rand((T,), generator=g, device=DEV).to(BF)
        self.wr, self.bias = (randn(g, E, H) * H ** -0.5).to(BF), randn(g, E) * 0.2
        self.w = [blocks("mx4", randn(g, E, *s) * s[1] ** -0.5) for s in ((F, H), (F, H), (H, F))]
        self.few = few

    def buffers(self):
        T, H = self.shape.T, self.shape.H
        o = {n: torch.full((T, H), float("nan"), dtype=BF, device=DEV) for n in ("s", "y", "s2", "y2")}
        o["q"], o["qs"] = (torch.zeros(T, n, dtype=torch.uint8, device=DEV) for n in (H, H // 32))
        o["layer"] = MoeLayerFew(self.shape, DEV, weights="mx4") if self.few else MoeLayerMx(self.shape, DEV, weight_bits=4)
        return o

    def run(self, o):
        s, L = self.shape, o["layer"]
        moe.moe_block_norm(s, self.x, EPS, residual=self.r, alpha=ALPHA, w_post=self.w_post, gate=self.gate, w_pre=self.w_pre,
                           s=o["s"], y=o["y"], q=o["q"], scales=o["qs"])
        if self.few:
            L.forward(o["y"], self.wr, self.bias, *self.w)
        else:
            moe.moe_router(s, o["y"], self.wr, self.bias, L.logits, L.ids, L.w, L.err, L.router_ws)
            L.experts(o["q"], o["qs"], L.ids, L.w, *self.w)
        moe.moe_block_norm(s, L.out, EPS, residual=o["s"], w_pre=self.w_last, s=o["s2"], y=o["y2"])

    def check(self, o):
        L = o["layer"]
        s, ds, _ = ref.block_norm(self.x, self.r, ALPHA, self.w_post, self.gate, 0, self.w_pre, EPS)
        ref.check(o["s"], (s, ds), "s", BF)
        ref.check(o["y"], ref.pre_norm(o["s"], self.w_pre, EPS)[:2], "y", BF)
        if self.few:
            check_few(L, o["y"], self.wr, self.bias, self.w, None, "layer")
        else:
            check_experts(L, o["q"], o["qs"], L.ids, self.w)
        s2, ds2, _ = ref.block_norm(L.out, o["s"], 1.0, None, None, 0, self.w_last, EPS)
        ref.check(o["s2"], (s2, ds2), "s2", BF)
        ref.check(o["y2"], ref.pre_norm(o["s2"], self.w_last, EPS)[:2], "y2", BF)


@pytest.mark.parametrize("T,H,E,k,F,few", [(1, 1024, 16, 4, 512, True), (19, 384, 8, 2, 256, True),
                                           (19, 384, 8, 2, 256, False), (333, 640, 12, 3, 384, False)])
def test_serving_step(T, H, E, k, F, few):
    step = Step(T, H, E, k, F, few, 100 + T)
    a, b, c = (step.buffers() for _ in range(3))
    step.run(a)
    torch.cuda.synchronize()
    step.check(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(b)
    side, g = torch.cuda.Stream(), gen(7)
    for i in range(4):
        step.x.copy_(randn(g, T, H))
        step.r.copy_(randn(g, T, H))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            step.run(c)
        torch.cuda.synchronize()
        step.run(a)
        torch.cuda.synchronize()
        for n in ("s", "y", "q", "qs", "s2", "y2"):
            assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n]), (i, n)
    step.check(a)


def test_the_two_layers_agree_on_the_same_weights():
    """A few tokens through both forms of the step: the same choice, and outputs apart
    by what the 8-bit rows and activations of one of them round: codes of half a step
    2^-4 in x and in h, each twice as a product's factor at worst by norm 2^-4 /
    sqrt(3) (0.036), together 0.036 sqrt(3) for x in gate, x in up and h (0.063)."""
    few, many = Step(19, 384, 8, 2, 256, True, 5), Step(19, 384, 8, 2, 256, False, 5)
    a, b = few.buffers(), many.buffers()
    few.run(a)
    many.run(b)
    torch.cuda.synchronize()
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["layer"].ids, b["layer"].ids)
    x, y = a["layer"].out.double(), b["layer"].out.double()
    assert float((x - y).norm() / x.norm()) <= 0.063


def stack64(x, W, w_post, gate, rows, w_pre):
    """The stream behind a stack of blocks y -> tanh(y W), float64, by autograd."""
    def norm(v, w):
        return v * (v.pow(2).mean(-1, keepdim=True) + EPS).rsqrt() * w

    s, y = x, norm(x, w_pre)
    for m in W:
        s = ALPHA * s + gate.repeat_interleave(rows, 0)[:x.shape[0]] * norm(torch.tanh(y @ m), w_post)
        y = norm(s, w_pre)
    return s, y


@pytest.mark.parametrize("T,H,rows", [(7, 96, 3), (1, 64, 1), (130, 256, 130)])
def test_gradient_of_a_stack_of_blocks(T, H, rows):
    """Three blocks that share the norms' weights and the gate. Each operator's error
    is at most some 60 roundings of float32 of its terms (2^-24 each), 14 operators
    follow each other, and gradients cancel to half of their terms: 14 * 60 * 2 *
    2^-24 = 1e-4, by norm."""
    g = gen(T + H)
    shape = moe.Shape(T, H, 1, 1, 64, 1, 0, moe.MOE_F32)
    x, co_s, co_y = (randn(g, T, H) for _ in range(3))
    W = [randn(g, H, H) * H ** -0.5 for _ in range(3)]
    w_post, w_pre = (1 + 0.2 * randn(g, H) for _ in range(2))
    gate = 0.5 + torch.rand((-(-T // rows), H), generator=g, device=DEV)
    leaves = [v.double().requires_grad_() for v in (x, w_post, gate, w_pre)]
    s, y = stack64(leaves[0], [m.double() for m in W], leaves[1], leaves[2], rows, leaves[3])
    want = torch.autograd.grad((s * co_s.double()).sum() + (y * co_y.double()).sum(), leaves)

    def new(*shape):
        return torch.full(shape, float("nan"), device=DEV)

    # forward: block i reads y[i], the stream is s[i]
    s, y, out, r1, r2 = [x], [new(T, H)], [], [], [new(T)]
    # (the first norm: a step without a residual, s = x)
    moe.moe_block_norm(shape, x, EPS, w_pre=w_pre, y=y[0], rstd_pre=r2[0])
    for m in W:
        out.append(torch.tanh(y[-1].double() @ m.double()).float())
        s.append(new(T, H)), y.append(new(T, H)), r1.append(new(T)), r2.append(new(T))
        moe.moe_block_norm(shape, out[-1], EPS, residual=s[-2], alpha=ALPHA, w_post=w_post, gate=gate, gate_rows=rows,
                           w_pre=w_pre, s=s[-1], y=y[-1], rstd_post=r1[-1], rstd_pre=r2[-1])
    # backward
    got = [None, torch.zeros(H, device=DEV), torch.zeros_like(gate), torch.zeros(H, device=DEV)]
    ds, dy = co_s.clone(), co_y.clone()
    for i in (2, 1, 0):
        ws = torch.empty(moe.moe_block_norm_backward_workspace_bytes(shape, rows), dtype=torch.uint8, device=DEV)
        dx, dw1, dg, dw2 = new(T, H), new(H), new(*gate.shape), new(H)
        moe.moe_block_norm_backward(shape, out[i], r1[i], dy, ds, dx, ws, s=s[i + 1], rstd_pre=r2[i + 1], alpha=ALPHA,
                                    w_post=w_post, gate=gate, gate_rows=rows, w_pre=w_pre, dresidual=ds, dw_post=dw1, dgate=dg,
                                    dw_pre=dw2)
        for to, v in zip(got[1:], (dw1, dg, dw2)):
            to += v
        t = out[i].double()
        dy = ((dx.double() * (1 - t * t)) @ W[i].double().t().contiguous()).float()
    ws = torch.empty(moe.moe_block_norm_backward_workspace_bytes(shape, 0), dtype=torch.uint8, device=DEV)
    dx, dw2 = new(T, H), new(H)
    moe.moe_block_norm_backward(shape, x, None, dy, ds, dx, ws, s=x, rstd_pre=r2[0], w_pre=w_pre, dw_pre=dw2)
    got[0], got[3] = dx, got[3] + dw2
    torch.cuda.synchronize()
    for n, a, b in zip(("x", "w_post", "gate", "w_pre"), got, want):
        off = float((a.double() - b).norm() / b.norm())
        print(n, off, flush=True)
        assert off <= 1e-4, (n, off)
