"""The calls of moe_block_norm and its backward that the header allows beside the whole
ones: every choice of outputs, every place that an output may share with an input, one
gradient alone and one array as both, on the kernels for all widths."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402

import step_ref as ref  # noqa: E402
from test_gpu_step import ALPHA, BF, DEV, EPS, F32, gen, randn, shape_of  # noqa: E402

pytestmark = pytest.mark.gpu


class Step:
    """Inputs of a step, its whole forward, and calls on them."""

    def __init__(self, T, H, t, rows, residual, post):
        g = gen(T + H)
        self.shape, self.t, self.rows = shape_of(T, H, t), t, rows
        self.x, self.r, self.dy, self.ds = (randn(g, T, H).to(t) for _ in range(4))
        self.w_post = (1 + 0.3 * randn(g, H)).to(t) if post else None
        self.w_pre = (1 + 0.3 * randn(g, H)).to(t)
        self.gate = (randn(g, T) if rows == 0 else randn(g, -(-T // rows), H)).to(t)
        self.residual = residual
        self.full = self.outputs()
        self.forward(**self.full)

    def outputs(self):
        T, H = self.x.shape
        o = dict(s=torch.empty_like(self.x), y=torch.empty_like(self.x), rstd_pre=torch.empty(T, device=DEV),
                 q=torch.empty(T, H, dtype=torch.uint8, device=DEV),
                 scales=torch.empty(T, H // 32, dtype=torch.uint8, device=DEV))
        if self.w_post is not None:
            o["rstd_post"] = torch.empty(T, device=DEV)
        return o

    def forward(self, x=None, r=None, pre=True, **outputs):
        moe.moe_block_norm(self.shape, self.x if x is None else x, EPS,
                           residual=(self.r if r is None else r) if self.residual else None, alpha=ALPHA, w_post=self.w_post,
                           gate=self.gate, gate_rows=self.rows, w_pre=self.w_pre if pre else None, **outputs)

    def backward(self, dy, ds, dx, dr, **outputs):
        ws = torch.full((moe.moe_block_norm_backward_workspace_bytes(self.shape, self.rows),), 0xFF, dtype=torch.uint8, device=DEV)
        only = dy is None   # (then nothing of the norm in front is read)
        moe.moe_block_norm_backward(self.shape, self.x, self.full.get("rstd_post"), dy, ds, dx, ws,
                                    s=None if only else self.full["s"], rstd_pre=None if only else self.full["rstd_pre"],
                                    alpha=ALPHA, w_post=self.w_post, gate=self.gate, gate_rows=self.rows,
                                    w_pre=None if only else self.w_pre, dresidual=dr, **outputs)


# one to four vectors a thread, one or two in the backward, and rows wider than the registers hold
STEPS = [(6, 4096, F32, 2), (3, 6144, F32, 2), (5, 640, BF, 0), (3, 96, F32, 1), (7, 12288, BF, 7), (3, 32832, BF, 1), (4, 20000, F32, 0)]


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T,H,t,rows", STEPS)
def test_forward(T, H, t, rows, residual, post):
    a = Step(T, H, t, rows, residual, post)
    for names in (["s"], ["y"], ["q", "scales"], ["rstd_pre"], ["rstd_post"], ["y", "rstd_pre"], ["s", "q", "scales"]):
        if post or "rstd_post" not in names:
            o = {n: v for n, v in a.outputs().items() if n in names}
            a.forward(**o)
            for n in o:
                assert torch.equal(o[n], a.full[n]), (names, n)
    s = torch.empty_like(a.x)
    a.forward(pre=False, s=s)
    assert torch.equal(s, a.full["s"])
    for s_in, y_in in (("x", None), (None, "x"), ("r", None), (None, "r"), ("x", "r"), ("r", "x")):
        d = {"x": a.x.clone(), "r": a.r.clone()}
        o = {n: d[into] for n, into in (("s", s_in), ("y", y_in)) if into and (residual or into == "x")}
        if o:
            a.forward(x=d["x"], r=d["r"], **o)
            for n in o:
                assert torch.equal(o[n], a.full[n]), (s_in, y_in, n)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("T,H,t,rows", STEPS)
def test_backward(T, H, t, rows, post):
    a = Step(T, H, t, rows, True, post)
    for dy, ds in ((a.dy, a.ds), (a.dy, None), (None, a.ds), (a.dy, a.dy)):
        dx, dr = torch.empty_like(a.x), torch.empty_like(a.x)
        sums = {"dgate": torch.empty(a.gate.shape, device=DEV)}
        if post:
            sums["dw_post"] = torch.empty(H, device=DEV)
        if dy is not None:
            sums["dw_pre"] = torch.empty(H, device=DEV)
        a.backward(dy, ds, dx, dr, **sums)
        want = ref.block_norm_bwd(a.x, a.full.get("rstd_post"), a.full["s"], a.full["rstd_pre"], ALPHA, a.w_post, a.gate, rows,
                                  a.w_pre, dy, ds)
        ref.check(dx, want["dx"], "dx", t)
        ref.check(dr, want["dresidual"], "dresidual", t)
        for n, v in sums.items():
            ref.check(v, want[n], n)
        # the two outputs in the gradients' places, either way round; and dx alone
        for turn in (False, True):
            g = [None if v is None else v.clone() for v in (dy, ds)]
            to = [torch.empty_like(a.x) if v is None else v for v in (g[::-1] if turn else g)]
            a.backward(*g, *to)
            assert torch.equal(to[0], dx) and torch.equal(to[1], dr), turn
        both = dy if dy is not None else ds
        both = both.clone()
        a.backward(both if dy is not None else None, both if dy is ds else ds, both, None)
        assert torch.equal(both, dx)
