"""Weight gradients in the largest tiles without splits: small whole numbers, so that every sum is exact, stored into and
added to gradients of each type."""
import pytest
import torch

from tests import rank_ops as R
from tests import weight_grad_plan as plan

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def zf():
    from fsdp_sharded_mixed_amd import zf as Z
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return Z


@pytest.fixture(autouse=True)
def _guards():
    R.Guarded.made = []
    yield
    R.check_guards()


@pytest.mark.parametrize("rows,outs,ins", plan.LARGE)
@pytest.mark.parametrize("dtype,grad_dtype", [(BF16, F32), (F16, F32), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("gap,skew", [(0, 0), (16, 1)])
def test_whole_numbers(zf, rows, outs, ins, dtype, grad_dtype, accumulate, gap, skew):
    """gap: elements between the rows of dy and of the codes.  skew: elements from an aligned address to the gradient's
    first one."""
    assert plan.chosen(rows, outs, ins) == ("big", 1)
    g = R.generator(rows + outs)
    dy = R.filled(torch.randint(-8, 9, (rows, outs), generator=g, device="cuda"), dtype, gap, 0, "dy")
    x = torch.randint(-8, 9, (rows, ins), generator=g, device="cuda").to(dtype)
    old = torch.randint(-8, 9, (outs, ins), generator=g, device="cuda").to(grad_dtype)
    grad = R.filled(old, grad_dtype, 0, skew, "grad")
    zf.weight_grad(dy, R.kept(zf, x, gap), grad, None, accumulate=accumulate)
    want = dy.double().t().contiguous() @ x.double() + (old.double() if accumulate else 0)
    assert float(want.abs().max()) < 2 ** 15  # exact in binary32, and in fp16's range
    assert torch.equal(grad, want.float().to(grad_dtype))
