"""Activation checkpoints in 8 bits against their definition, bit for bit."""
import pytest
import torch

from tests import rank_ops as R

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


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


def check(zf, x, gap=0, skew=0):
    """Stores x and loads it back; both against the definition."""
    a = R.blank(zf, *x.shape, gap, skew)
    zf.act8_store(a, x)
    codes, scales = R.keep(x)
    assert torch.equal(a.scales, scales)
    assert torch.equal(a.codes, codes)
    for dtype in TYPES:
        back = R.buffer(*x.shape, dtype, gap, skew, "loaded")
        zf.act8_load(a, back)
        want = R.numbers(codes, scales).to(dtype)
        assert torch.equal(back.isnan(), want.isnan())
        assert torch.equal(back[~want.isnan()], want[~want.isnan()])
    return a


def spread(g, rows, cols, dtype):
    """Activations over many orders of magnitude, a zero here and there."""
    x = R.normal(g, rows, cols) * torch.exp2(torch.randint(-12, 10, (rows, -(-cols // 32)), generator=g, device="cuda")
                                             .float().repeat_interleave(32, 1)[:, :cols])
    return (x * (R.normal(g, rows, cols).abs() > 0.1)).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,gap,skew", [
    (1, 1, 0, 0), (1, 31, 0, 1), (3, 32, 1, 3), (2, 33, 0, 0), (5, 64, 8, 0), (7, 95, 1, 1), (4, 1000, 3, 5),
    (130, 2048, 0, 0), (33, 2049, 0, 1), (9, 8192, 16, 0), (3, 20001, 0, 0), (1025, 8, 0, 0)])
def test_sizes(zf, dtype, rows, cols, gap, skew):
    x = R.filled(spread(R.generator(rows * 31 + cols), rows, cols, dtype), dtype, gap, skew, "x")
    check(zf, x, gap, skew)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_16_bit_pattern(zf, dtype):
    """All 65536 patterns, alone in their groups, and beside each power of two that a group may hold."""
    every = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(dtype)
    alone = torch.zeros(65536, 2, dtype=dtype, device="cuda")
    alone[:, 0] = every
    check(zf, alone)
    for power in range(-20, 16, 5):
        beside = alone.clone()
        beside[:, 1] = 2.0 ** power
        check(zf, beside)
    check(zf, every.view(1, -1).contiguous())  # neighbouring patterns in one group
    check(zf, every[torch.randperm(65536, generator=R.generator(1), device="cuda")].view(64, 1024))


def test_every_code_with_every_scale(zf):
    """256 codes and the 221 scales that a store writes: exact in fp32 and bf16, rounded once in fp16."""
    codes = torch.arange(256, device="cuda").to(torch.uint8).repeat(221, 1)
    scales = torch.arange(27, 248, device="cuda").to(torch.uint8).view(-1, 1).repeat(1, 8).contiguous()
    want = R.numbers(codes, scales)
    for dtype in TYPES:
        out = R.buffer(221, 256, dtype)
        zf.act8_load(zf.act8(codes, scales), out)
        exact = want.to(torch.float32).to(dtype) if dtype == torch.float16 else want.to(dtype)
        assert torch.equal(out.isnan(), want.isnan())
        assert torch.equal(out[~want.isnan()], exact[~want.isnan()])


def test_fp32_extremes(zf):
    """The largest and smallest numbers, borders of the scale, infinities and NaN in every place of a group."""
    m = torch.finfo(torch.float32).max
    values = [m, -m, 1.9375 * 2.0 ** 127, 1.75 * 2.0 ** 127, 2.0 ** -126, 2.0 ** -149, 448.0, 448.00003, 2.0 ** -93, 2.0 ** -92,
              1.75 * 2.0 ** -92, 0.0, -0.0, 2.0 ** -110, 447.99997, 464.0, 1e-30]
    x = torch.zeros(len(values) + 64, 64, device="cuda")
    for i, v in enumerate(values):
        x[i, i] = v
        x[i, 40] = v
        x[i, 41] = v / 3
    for i in range(64):
        x[len(values) + i] = torch.linspace(-3, 3, 64)
        x[len(values) + i, i] = (float("inf"), float("nan"), -float("inf"))[i % 3]
    check(zf, x)
    check(zf, x.to(torch.bfloat16))


def test_no_rows(zf):
    a = zf.act8(torch.empty(0, 64, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, dtype=torch.uint8, device="cuda"))
    zf.act8_store(a, torch.empty(0, 64, device="cuda"))
    zf.act8_load(a, torch.empty(0, 64, device="cuda"))


def test_many_rows(zf):
    """More rows than a launch has blocks for at once."""
    x = R.normal(R.generator(4), (1 << 22) * 64 + 77, 8).to(torch.bfloat16)
    a = zf.act8(torch.empty(*x.shape, dtype=torch.uint8, device="cuda"),
                torch.empty(x.shape[0], 1, dtype=torch.uint8, device="cuda"))
    zf.act8_store(a, x)
    back = torch.empty_like(x)
    zf.act8_load(a, back)
    for part in (slice(0, 5000), slice(x.shape[0] // 2, x.shape[0] // 2 + 5000), slice(-5000, None)):
        codes, scales = R.keep(x[part])
        assert torch.equal(a.codes[part], codes) and torch.equal(a.scales[part], scales)
        assert torch.equal(back[part].double(), R.numbers(codes, scales))
    assert bool(((back - x).abs() <= x.abs() / 16 + 2.0 ** -9).all())
