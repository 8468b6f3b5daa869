"""Ways of calling the operators around the layer (include/moe_block.h) on the
GPU that the other tests do not take."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402
from expert_load_balance_amd.layer import MoeLayerMx  # noqa: E402

from test_gpu_block import DEV, gen, model, run_step, step_inputs  # noqa: E402

pytestmark = pytest.mark.gpu


def test_serving_step_on_a_raw_stream_handle():
    """A stream may be given as its handle, as to every call of the package."""
    shape = moe.Shape(20, 512, 8, 2, 384, 4, 1, moe.MOE_BF16)
    g = gen(5)
    m, inp = model(g, shape), step_inputs(g, shape)
    L = MoeLayerMx(shape, DEV)
    want = run_step(L, inp, m)[0].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side.cuda_stream, torch.cuda.default_stream().cuda_stream, side):
        L.out.zero_()
        L.err.fill_(moe.ERR_RANGE)             # cleared by the step, on its stream
        torch.cuda.synchronize()
        got = run_step(L, inp, m, stream=st)[0]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and int(L.err.item()) == 0
