"""The numbers that a weight gradient's products take: each code with each scale in dy's type, and every dy.  One token
has one product a result, so results are known to the bit."""
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


def same(got, want):
    """Equal numbers, infinities and NaN in the same places."""
    assert torch.equal(got.isnan(), want.isnan())
    bad = ~got.isnan() & (got.double() != want.double())
    assert not bool(bad.any()), [(i, float(got.flatten()[i]), float(want.flatten()[i]))
                                 for i in bad.flatten().nonzero()[:8, 0].tolist()]


def one_token(zf, codes, scales, dy, skew):
    c, s = R.buffer(*codes.shape, torch.uint8, 0, skew, "codes"), R.buffer(*scales.shape, torch.uint8, 0, skew, "scales")
    c.copy_(codes)
    s.copy_(scales)
    dy = R.filled(dy, dy.dtype, 0, skew, "dy")
    outs, ins = dy.shape[1], codes.shape[1]
    grad = R.buffer(outs, ins, F32, 0, skew, "grad")
    zf.weight_grad(dy, zf.act8(c, s), grad, R.bytes_buffer(max(1, zf.weight_grad_bytes(1, outs, ins))))
    return grad


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("skew", [0, 1])
def test_every_code_with_every_scale(zf, dtype, skew):
    """256 codes with the 221 scales that a store writes, as numbers of dy's type: bf16 holds them; fp16 rounds them to
    nearest even, subnormals among them, and past its largest number they are infinities.  (Codes above 240 at the
    largest scale, which no store writes, are left out.)"""
    codes = torch.arange(256, device="cuda").to(torch.uint8).repeat(221, 1)
    codes[-1] = torch.where((codes[-1] & 127 > 119) & (codes[-1] & 127 < 127), 119, codes[-1])
    scales = torch.arange(27, 248, device="cuda").to(torch.uint8).view(-1, 1).repeat(1, 8).contiguous()
    numbers = R.numbers(codes, scales).view(1, -1)
    dy = torch.tensor([[1.0, -0.5, 0.25]], device="cuda").to(dtype)
    grad = one_token(zf, codes.view(1, -1), scales.view(1, -1), dy, skew)
    want = numbers.float().to(dtype).double() * dy.double().t()
    same(grad, want)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("scale", [120, 140])
def test_every_gradient(zf, dtype, scale):
    """All 65536 patterns of dy, subnormals and what is not finite among them, times 2^-7 or 2^13 (code 56 is 1)."""
    dy = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(dtype).view(1, -1)
    codes, scales = torch.full((1, 40), 56, device="cuda"), torch.full((1, 2), scale, device="cuda")
    grad = one_token(zf, codes.to(torch.uint8), scales.to(torch.uint8), dy, 0)
    want = (dy.double().t() * 2.0 ** (scale - 127)).expand(65536, 40)
    same(grad, want.float())


def whole(g, rows, cols, dtype, stride):
    """Whole numbers from -8 to 8 in rows that lie `stride` elements apart, the elements between them never written."""
    full = torch.empty((rows - 1) * stride + cols, dtype=dtype, device="cuda")
    t = torch.as_strided(full, (rows, cols), (stride, 1))
    return t.copy_(torch.randint(-8, 9, (rows, cols), generator=g, device="cuda"))


@pytest.mark.parametrize("dy_bytes,code_bytes", [(0, 0), (-16, 0), (0, -16), (-16, -16)])
def test_the_longest_strides_of_whole_pieces(zf, dy_bytes, code_bytes):
    """Rows of gradients and of codes 2^24 bytes apart, and 16 bytes less: 128 of the latter fit an offset of 31 bits,
    so they go straight to shared memory, and the former through registers."""
    g = R.generator(20)
    rows, outs, ins = 161, 200, 272
    dy = whole(g, rows, outs, BF16, (2 ** 24 + dy_bytes) // 2)
    x = whole(g, rows, ins, BF16, ins)
    codes, scales = R.keep(x)
    far = torch.as_strided(torch.empty((rows - 1) * (2 ** 24 + code_bytes) + ins, dtype=torch.uint8, device="cuda"),
                           (rows, ins), (2 ** 24 + code_bytes, 1)).copy_(codes)
    grad = R.buffer(outs, ins, F32, what="grad")
    zf.weight_grad(dy, zf.act8(far, scales), grad, R.bytes_buffer(max(1, zf.weight_grad_bytes(rows, outs, ins))))
    assert torch.equal(grad.double(), dy.double().t().contiguous() @ x.double())
    del dy, far
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
