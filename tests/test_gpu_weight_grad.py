"""A Linear's weight gradient from its input's checkpoint against the product in 64 bits.

Bounds.  Products of a 16-bit gradient and a checkpoint's number are exact in binary32 up to its rounding; a sum over n
tokens takes n additions, each off by at most one unit of binary32 (2 U32), whatever the matrix instruction's order."""
import pytest
import torch

from tests import rank_ops as R

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


def check(zf, x, dy, grad_dtype, accumulate, gap=0, skew=0):
    rows, outs = dy.shape
    ins = x.shape[1]
    a = R.kept(zf, x, gap, skew)
    grad = R.filled(R.normal(R.generator(2), outs, ins), grad_dtype, 0, skew, "grad")
    old = grad.clone()
    ws = R.bytes_buffer(max(1, zf.weight_grad_bytes(rows, outs, ins)))
    zf.weight_grad(dy, a, grad, ws, accumulate=accumulate)
    xv = R.numbers(*R.keep(x)).to(dy.dtype).double()
    total = dy.double().t().contiguous() @ xv
    size = dy.double().abs().t().contiguous() @ xv.abs()
    R.assert_within(grad, *R.written(total, (rows + 8) * 2 * R.U32 * size, old, grad_dtype, accumulate), "grad")
    return grad


SIZES = [(1, 1, 1, 0, 0), (1, 16, 32, 0, 0), (3, 5, 7, 1, 1), (64, 128, 128, 0, 0), (65, 129, 127, 0, 1),
         (100, 40, 333, 3, 1), (333, 777, 1000, 0, 0), (1000, 130, 70, 8, 0), (63, 257, 513, 0, 3), (2048, 64, 64, 0, 0),
         (4100, 256, 272, 16, 0), (130, 1024, 512, 0, 0), (700, 8, 2000, 0, 0), (257, 520, 776, 8, 8)]


@pytest.mark.parametrize("dtype,grad", [(BF16, F32), (BF16, BF16), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,outs,ins,gap,skew", SIZES)
def test_sizes(zf, dtype, grad, accumulate, rows, outs, ins, gap, skew):
    g = R.generator(rows + outs * 3 + ins)
    x = R.normal(g, rows, ins).to(dtype)
    dy = R.filled(R.normal(g, rows, outs) * 0.1, dtype, gap, skew, "dy")
    check(zf, x, dy, grad, accumulate, gap, skew)


def test_a_large_one(zf):
    g = R.generator(4)
    check(zf, R.normal(g, 3000, 2048).to(BF16), R.filled(R.normal(g, 3000, 1536), BF16), F32, False)
    check(zf, R.normal(g, 8192, 1024).to(F16), R.filled(R.normal(g, 8192, 1000), F16), F32, True)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_whole_numbers_are_exact(zf, dtype):
    """Small whole numbers: every product and sum is exact, so every place is in its place."""
    g = R.generator(9)
    for rows, outs, ins in ((512, 300, 200), (70, 64, 1000), (200, 520, 264)):
        x = torch.randint(-8, 9, (rows, ins), generator=g, device="cuda").to(dtype)
        dy = torch.randint(-8, 9, (rows, outs), generator=g, device="cuda").to(dtype)
        grad = torch.empty(outs, ins, device="cuda")
        zf.weight_grad(dy, R.kept(zf, x), grad, R.bytes_buffer(max(1, zf.weight_grad_bytes(rows, outs, ins))))
        assert torch.equal(grad.double(), dy.double().t().contiguous() @ x.double())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,outs,ins", [(40, 2056, 2320), (70, 2049, 2051), (1, 2200, 2000), (600, 2100, 2064),
                                           (8200, 1104, 1200), (8200, 1101, 1201), (6200, 2056, 2064), (6200, 2049, 2062)])
def test_whole_numbers_are_exact_in_large_tiles(zf, dtype, rows, outs, ins):
    """Sizes that larger tiles take, with and without whole pieces and with tokens split over blocks: sums stay below
    2^24, so every place holds the exact number."""
    g = R.generator(10)
    x = torch.randint(-8, 9, (rows, ins), generator=g, device="cuda").to(dtype)
    dy = torch.randint(-8, 9, (rows, outs), generator=g, device="cuda").to(dtype)
    grad = torch.ones(outs, ins, device="cuda")
    ws = R.bytes_buffer(max(1, zf.weight_grad_bytes(rows, outs, ins)))
    zf.weight_grad(dy, R.kept(zf, x), grad, ws, accumulate=True)
    want = dy.float().t().contiguous().double() @ x.double() + 1
    assert torch.equal(grad.double(), want)


@pytest.mark.parametrize("gap,skew", [(0, 0), (1, 1), (5, 3)])
@pytest.mark.parametrize("rows,outs,ins", [(700, 1, 1), (3000, 5, 3), (5001, 63, 127), (5001, 64, 128), (2500, 65, 129),
                                           (1025, 129, 500), (2500, 2051, 2053)])
def test_whole_numbers_are_exact_in_odd_rows(zf, rows, outs, ins, gap, skew):
    """Rows shorter and longer than a tile, at any alignment: pieces that end past their row, and past the matrix."""
    g = R.generator(11)
    x = torch.randint(-8, 9, (rows, ins), generator=g, device="cuda").to(F16)
    dy = R.filled(torch.randint(-8, 9, (rows, outs), generator=g, device="cuda"), F16, gap, skew, "dy")
    grad = torch.empty(outs, ins, device="cuda")
    ws = R.bytes_buffer(max(1, zf.weight_grad_bytes(rows, outs, ins)))
    zf.weight_grad(dy, R.kept(zf, x, gap, skew), grad, ws)
    assert torch.equal(grad.double(), dy.float().t().contiguous().double() @ x.double())


def test_scales_far_apart(zf):
    """Groups whose scales differ by many powers of two, tiny and huge ones among them."""
    g = R.generator(10)
    x = R.normal(g, 96, 320) * torch.exp2(torch.randint(-60, 60, (96, 10), generator=g, device="cuda").float()
                                          .repeat_interleave(32, 1))
    check(zf, x.to(BF16), R.filled(R.normal(g, 96, 100), BF16), F32, False)
    small = R.normal(g, 96, 320) * torch.exp2(torch.randint(-20, 8, (96, 10), generator=g, device="cuda").float()
                                              .repeat_interleave(32, 1))
    check(zf, small.to(F16), R.filled(R.normal(g, 96, 100), F16), F32, False)


def test_what_is_not_finite_stays_in_its_row_and_column(zf):
    g = R.generator(11)
    x, dy = R.normal(g, 70, 200).to(BF16), R.normal(g, 70, 150).to(BF16)
    want = torch.empty(150, 200, device="cuda")
    ws = R.bytes_buffer(max(1, zf.weight_grad_bytes(70, 150, 200)))
    zf.weight_grad(dy, R.kept(zf, x), want, ws)
    x[3, 17], x[69, 150], dy[5, 40] = float("nan"), float("inf"), float("nan")
    codes, scales = R.keep(torch.where(torch.isfinite(x), x, 0.0).to(BF16))
    codes[3, 17] = codes[69, 150] = 127
    grad = torch.empty_like(want)
    zf.weight_grad(dy, zf.act8(codes, scales), grad, ws)
    hit = torch.zeros(150, 200, dtype=torch.bool, device="cuda")
    hit[:, 17] = hit[:, 150] = hit[40] = True
    assert torch.equal(grad.isnan(), hit)


def test_no_rows(zf):
    dy, a = torch.empty(0, 8, dtype=BF16, device="cuda"), R.blank(zf, 0, 40)
    grad = R.filled(torch.ones(8, 40, device="cuda"), F32)
    zf.weight_grad(dy, a, grad, None, accumulate=True)
    assert bool((grad == 1).all())
    zf.weight_grad(dy, a, grad, None)
    assert bool((grad == 0).all())


def test_the_same_call_gives_the_same_bits(zf):
    g = R.generator(6)
    x, dy = R.normal(g, 5000, 200).to(BF16), R.normal(g, 5000, 300).to(BF16)
    a, got = R.kept(zf, x), []
    ws = R.bytes_buffer(max(1, zf.weight_grad_bytes(5000, 300, 200)))
    for k in range(3):
        ws.fill_(0x21 * k)
        got.append(torch.empty(300, 200, device="cuda"))
        zf.weight_grad(dy, a, got[-1], ws)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_gradient_against_differences(zf):
    """The loss sum(dy * (x W^T)) is linear in W: its change along a direction is the gradient's product with it."""
    g = R.generator(13)
    x, dy = R.normal(g, 90, 64).to(BF16), R.normal(g, 90, 48).to(BF16)
    grad = torch.empty(48, 64, device="cuda")
    zf.weight_grad(dy, R.kept(zf, x), grad, R.bytes_buffer(max(1, zf.weight_grad_bytes(90, 48, 64))))
    xv, to = R.numbers(*R.keep(x)), R.normal(g, 48, 64).double()

    def loss(w):
        return float((dy.double() * (xv @ w.t().contiguous())).sum())
    change = (loss(to) - loss(-to)) / 2
    terms = float((dy.double().abs() * (xv.abs() @ to.abs().t().contiguous())).sum())
    assert abs(float((grad.double() * to).sum()) - change) <= terms * 200 * R.U32
