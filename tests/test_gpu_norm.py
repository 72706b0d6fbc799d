"""Layer norm and RMS norm, their checkpoints and their gradients against the formulas in 64 bits.

Bounds.  A row's sum in binary32 is a chain of at most d additions (the terms of a lane, then a tree over lanes and
waves), so it is off by d U32 times the sum of magnitudes; products and the rest count their roundings."""
import pytest
import torch

from tests import rank_ops as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5
U = R.U32


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


def depth(cols):
    return 80 + cols // 256


def vector(g, cols, dtype, skew, around):
    return R.filled(around + 0.3 * R.normal(g, 1, cols), dtype, 0, skew, "parameter").view(-1)


def statistics(x, kind, eps=EPS):
    """mean, 1 / sqrt(var + eps) and their bounds for binary32."""
    cols, x = x.shape[1], x.double()
    d = depth(cols)
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros(len(x), 1, dtype=torch.float64, device=x.device)
    off_mean = (d + 2) * U * x.abs().mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(mean)
    away = x - mean
    var = away.square().mean(1, keepdim=True)
    # each term's distance is off by off_mean and a rounding; the sum by its chain
    size = (away.abs() + off_mean).square().mean(1, keepdim=True)
    off_var = (d + 6) * U * size + (off_mean + U * (away.abs() + off_mean).mean(1, keepdim=True)) ** 2 \
        + 2 * U * size
    rstd = (var + eps).rsqrt()
    off_rstd = rstd * (0.5 * off_var / (var + eps) * 1.01 + 4 * U)
    return mean, off_mean, rstd, off_rstd


def check_forward(zf, kind, x, w, b, keep, y=None, gap=0, skew=0, eps=EPS):
    rows, cols = x.shape
    y = R.buffer(rows, cols, x.dtype, gap, skew, "y") if y is None else y
    x0 = x.clone()
    mean = R.buffer(1, rows, F32, 0, 1, "mean").view(-1) if kind == "layer" else None
    rstd = R.buffer(1, rows, F32, 0, 1, "rstd").view(-1)
    x8 = R.blank(zf, rows, cols, gap, skew) if "x" in keep else None
    y8 = R.blank(zf, rows, cols, 0, skew) if "y" in keep else None
    zf.layer_norm(zf.NORM_LAYER if kind == "layer" else zf.NORM_RMS, x, w, b, eps, y, mean, rstd, x8=x8, y8=y8)
    m, off_m, r, off_r = statistics(x0, kind, eps)
    if kind == "layer":
        R.assert_within(mean, m[:, 0], off_m[:, 0] + U * m[:, 0].abs(), "mean")
    R.assert_within(rstd, r[:, 0], off_r[:, 0], "rstd")
    away, wd = x0.double() - m, w.double().abs()
    want = away * r * w.double() + (b.double() if b is not None else 0)
    error = wd * ((away.abs() + off_m) * (off_r + 3 * U * r) + off_m * r)
    if b is not None:
        error = error + (want.abs() + error) * U
    R.assert_within(y, want, R.rounded(want, error * 1.01, x.dtype), "y")
    for a, v in ((x8, x0), (y8, y)):
        if a is not None:
            codes, scales = R.keep(v)
            assert torch.equal(a.scales, scales) and torch.equal(a.codes, codes)
    return y, mean, rstd


SIZES = [(1, 1, 0, 0), (3, 2, 1, 1), (5, 7, 0, 1), (17, 40, 0, 0), (33, 128, 8, 0), (6, 129, 1, 3), (9, 512, 0, 0),
         (4, 777, 0, 1), (13, 1024, 0, 0), (5, 1500, 3, 1), (8, 2048, 0, 0), (3, 2049, 0, 0), (2, 4096, 8, 0),
         (3, 5001, 0, 1), (2, 8192, 0, 0), (2, 10000, 1, 1), (1, 16384, 0, 0), (2, 16385, 0, 1), (2, 40001, 0, 0)]


@pytest.mark.parametrize("kind", R.KINDS)
@pytest.mark.parametrize("dtype,wdtype,bias,keep", [(BF16, BF16, True, "xy"), (BF16, F32, False, "y"),
                                                    (F16, F16, True, "x"), (F32, F32, False, "xy"), (F32, BF16, True, "")])
@pytest.mark.parametrize("rows,cols,gap,skew", SIZES)
def test_forward(zf, kind, dtype, wdtype, bias, keep, rows, cols, gap, skew):
    g = R.generator(rows + cols)
    x = R.filled(R.normal(g, rows, cols) * 3 + R.normal(g, rows, 1), dtype, gap, skew, "x")
    w = vector(g, cols, wdtype, skew, 1.0)
    b = vector(g, cols, wdtype, skew, 0.0) if bias else None
    check_forward(zf, kind, x, w, b, keep, None, gap, skew)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("cols", [3, 60, 64, 100, 520, 300, 1032, 2000, 2056, 4104, 4100, 9000, 9001, 16392, 17000])
def test_a_mean_whose_product_with_rstd_no_number_holds(zf, kept, cols):
    """x = mean = 2^120 in every element and rstd = 1000: x - mean is 0 and -mean * rstd is not finite, so lanes behind a
    row's end may not take part.  dx = rstd (h - avg(h)), weight_grad = 0, bias_grad = the sum of dy."""
    g = R.generator(cols)
    rows = 9
    x = torch.full((rows, cols), 2.0 ** 120, device="cuda")
    mean, rstd = torch.full((rows,), 2.0 ** 120, device="cuda"), torch.full((rows,), 1000.0, device="cuda")
    dy, w = R.filled(R.normal(g, rows, cols), F32), vector(g, cols, F32, 0, 1.0)
    dx = R.buffer(rows, cols, F32)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = R.bytes_buffer(zf.layer_norm_grad_bytes(rows, cols))
    zf.layer_norm_grad(zf.NORM_LAYER, dy, R.kept(zf, x) if kept else x, w, mean, rstd, dx, dw, db, ws)
    h = dy.double() * w.double()
    want = 1000.0 * (h - h.mean(1, keepdim=True))
    # h one rounding, its sum a chain, the mean and the difference one each, and the product
    off = (depth(cols) + 3) * U * h.abs().mean(1, keepdim=True) + 3 * U * (h.abs() + h.mean(1, keepdim=True).abs())
    R.assert_within(dx, want, 1000.0 * off * 1.01 + U * want.abs(), "dx")
    assert bool((dw == 0).all())
    R.assert_within(db, dy.double().sum(0), rows * U * dy.double().abs().sum(0), "bias_grad")


@pytest.mark.parametrize("cols", [100, 2048, 6000, 20000])
def test_a_mean_far_from_zero(zf, cols):
    """Rows around 1000 with unit deviation: the variance is that of the distances, not a difference of sums."""
    g = R.generator(cols)
    x = R.filled(R.normal(g, 40, cols) + 1000.0, F32)
    check_forward(zf, "layer", x, vector(g, cols, F32, 0, 1.0), None, "")


@pytest.mark.parametrize("kind", R.KINDS)
@pytest.mark.parametrize("cols", [64, 1000, 3000, 17000])
def test_in_place(zf, kind, cols):
    g = R.generator(cols)
    x = R.filled(R.normal(g, 21, cols), BF16, 8)
    check_forward(zf, kind, x, vector(g, cols, BF16, 0, 1.0), None, "xy", x, 0, 0)


@pytest.mark.parametrize("kind", R.KINDS)
@pytest.mark.parametrize("cols", [40, 1000, 5000, 20000])
def test_rows_without_values(zf, kind, cols):
    """A row of zeros, a constant row, infinities and NaN: each stays in its row."""
    g = R.generator(cols)
    x = R.normal(g, 9, cols)
    x[1], x[2], x[3, 5], x[4, 7], x[5, 0] = 0.0, 2.5, float("inf"), float("nan"), -float("inf")
    x, w = R.filled(x, F32), vector(g, cols, F32, 0, 1.0)
    y, mean = R.buffer(9, cols, F32), R.buffer(1, 9, F32).view(-1) if kind == "layer" else None
    rstd, x8 = R.buffer(1, 9, F32).view(-1), R.blank(zf, 9, cols)
    zf.layer_norm(zf.NORM_LAYER if kind == "layer" else zf.NORM_RMS, x, w, None, EPS, y, mean, rstd, x8=x8)
    codes, scales = R.keep(x)
    assert torch.equal(x8.codes, codes) and torch.equal(x8.scales, scales)
    fine = torch.tensor([True, True, True, False, False, False, True, True, True], device="cuda")
    assert bool(torch.isfinite(y[fine]).all()) and bool((y[1] == 0).all())
    if kind == "layer":
        assert bool((~torch.isfinite(y[~fine])).all()) and bool((y[2].abs() <= 1e-3).all())
    else:  # 1 / sqrt(inf) is 0: an infinity's row is zeros beside inf * 0
        assert bool(y[3, 5].isnan() and (y[3, :5] == 0).all() and y[4].isnan().all())
    kept_rows = torch.arange(9, device="cuda")[fine]
    alone = R.buffer(len(kept_rows), cols, F32)
    zf.layer_norm(zf.NORM_LAYER if kind == "layer" else zf.NORM_RMS, x[kept_rows].contiguous(), w, None, EPS, alone,
                  torch.empty(6, device="cuda") if kind == "layer" else None, torch.empty(6, device="cuda"))
    assert torch.equal(alone, y[kept_rows])


def gradients(kind, x, dy, w, mean, rstd):
    """dx, dw, db in 64 bits from given statistics, and bounds for binary32 before the results' rounding."""
    rows, cols = x.shape
    x, dy, w, r = x.double(), dy.double(), w.double(), rstd.double()[:, None]
    m = mean.double()[:, None] if kind == "layer" else torch.zeros_like(r)
    d = depth(cols)
    xh, h = (x - m) * r, dy * w
    off_xh = 2 * U * xh.abs()
    c1 = h.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(r)
    off_c1 = (d + 4) * U * h.abs().mean(1, keepdim=True) if kind == "layer" else c1
    c2, off_c2 = (h * xh).mean(1, keepdim=True), (d + 7) * U * (h * xh).abs().mean(1, keepdim=True)
    dx = r * (h - c1 - xh * c2)
    error = r * (4 * U * (h.abs() + c1.abs() + (xh * c2).abs()) + off_c1 + xh.abs() * off_c2
                 + off_xh * (c2.abs() + off_c2)) * 1.01
    dw, db = (dy * xh).sum(0), dy.sum(0)
    off_dw = (rows + 6) * U * (dy * xh).abs().sum(0)
    off_db = (rows + 3) * U * dy.abs().sum(0)
    return dx, error, dw, off_dw, db, off_db


def check_backward(zf, kind, x, dy, w, grad_dtype, bias, accumulate, kept, dx=None, gap=0, skew=0, weight=True):
    rows, cols = dy.shape
    g = R.generator(99)
    mean64, _, rstd64, _ = statistics(x, kind)
    mean = mean64.float().view(-1) if kind == "layer" else None
    rstd = rstd64.float().view(-1)
    dx = R.buffer(rows, cols, dy.dtype, gap, skew, "dx") if dx is None else dx
    dw = R.filled(R.normal(g, 1, cols), grad_dtype, 0, skew, "dw").view(-1) if weight else None
    db = R.filled(R.normal(g, 1, cols), grad_dtype, 0, skew, "db").view(-1) if bias else None
    old_w, old_b = (t.clone() if t is not None else None for t in (dw, db))
    given = R.kept(zf, x, gap, skew) if kept else x
    xv = R.numbers(*R.keep(x)) if kept else x
    want = gradients(kind, xv, dy.clone(), w, mean, rstd)
    ws = R.bytes_buffer(zf.layer_norm_grad_bytes(rows, cols)) if weight or bias else None
    zf.layer_norm_grad(zf.NORM_LAYER if kind == "layer" else zf.NORM_RMS, dy, given, w, mean, rstd, dx, dw, db, ws,
                       accumulate=accumulate)
    R.assert_within(dx, want[0], R.rounded(want[0], want[1], dx.dtype), "dx")
    for got, old, total, error, what in ((dw, old_w, want[2], want[3], "dw"), (db, old_b, want[4], want[5], "db")):
        if got is not None:
            R.assert_within(got, *R.written(total, error, old, grad_dtype, accumulate), what)
    return dx, dw, db


@pytest.mark.parametrize("kind", R.KINDS)
@pytest.mark.parametrize("dtype,wdtype,gdtype,bias,accumulate,kept", [
    (BF16, BF16, F32, True, True, False), (BF16, BF16, BF16, False, False, True), (F16, F16, F16, True, False, False),
    (BF16, F32, F32, False, True, True), (F32, F32, F32, True, False, True), (F16, F32, F16, True, True, True)])
@pytest.mark.parametrize("rows,cols,gap,skew", SIZES + [(700, 40, 0, 0), (1025, 130, 0, 0), (300, 2048, 0, 0),
                                                        (257, 3001, 0, 1), (90, 17000, 0, 0)])
def test_backward(zf, kind, dtype, wdtype, gdtype, bias, accumulate, kept, rows, cols, gap, skew):
    g = R.generator(rows * 3 + cols)
    x = R.filled(R.normal(g, rows, cols) * 2 + R.normal(g, rows, 1), dtype, gap, skew, "x")
    dy = R.filled(R.normal(g, rows, cols) * 0.1, dtype, gap, skew, "dy")
    check_backward(zf, kind, x, dy, vector(g, cols, wdtype, skew, 1.0), gdtype, bias, accumulate, kept, None, gap, skew)


@pytest.mark.parametrize("kind", R.KINDS)
@pytest.mark.parametrize("cols", [100, 1000, 4000, 17000])
def test_backward_in_place_and_frozen(zf, kind, cols):
    """dx in dy's place; no gradient of the parameters wanted, or of the bias alone."""
    g = R.generator(cols)
    x, w = R.filled(R.normal(g, 30, cols), BF16), vector(g, cols, BF16, 0, 1.0)
    for weight, bias in ((False, False), (False, True), (True, False)):
        dy = R.filled(R.normal(g, 30, cols), BF16, 3)
        check_backward(zf, kind, x, dy, w, F32, bias, False, False, dy, weight=weight)


def test_many_rows(zf):
    """Thousands of rows a block, and partial sums of every block."""
    g = R.generator(5)
    for rows, cols in ((40000, 24), (20000, 200), (9000, 2100)):
        x, dy = R.filled(R.normal(g, rows, cols), BF16), R.filled(R.normal(g, rows, cols), BF16)
        check_backward(zf, "layer", x, dy, vector(g, cols, BF16, 0, 1.0), F32, True, False, False)


def test_no_rows(zf):
    w, none = torch.ones(64, device="cuda"), torch.empty(0, 64, device="cuda")
    stat = torch.empty(0, device="cuda")
    zf.layer_norm(zf.NORM_RMS, none, w, None, EPS, torch.empty_like(none), None, stat)
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    ws = R.bytes_buffer(zf.layer_norm_grad_bytes(0, 64))
    zf.layer_norm_grad(zf.NORM_RMS, none, none, w, None, stat, torch.empty_like(none), dw, db, ws, accumulate=True)
    assert bool((dw == 1).all() and (db == 1).all())
    zf.layer_norm_grad(zf.NORM_RMS, none, none, w, None, stat, torch.empty_like(none), dw, db, ws)
    assert bool((dw == 0).all() and (db == 0).all())


def test_the_same_call_gives_the_same_bits(zf):
    g = R.generator(6)
    x, dy, w = (R.normal(g, 3000, 1000), R.normal(g, 3000, 1000), R.normal(g, 1000))
    mean, rstd, y = torch.empty(3000, device="cuda"), torch.empty(3000, device="cuda"), torch.empty_like(x)
    zf.layer_norm(zf.NORM_LAYER, x, w, None, EPS, y, mean, rstd)
    ws, got = R.bytes_buffer(zf.layer_norm_grad_bytes(3000, 1000)), []
    for k in range(3):
        ws.fill_(0x33 * k)
        got.append([torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)])
        zf.layer_norm_grad(zf.NORM_LAYER, dy, x, w, mean, rstd, *got[-1], ws)
    for k in (1, 2):
        assert all(torch.equal(a, b) for a, b in zip(got[0], got[k]))


@pytest.mark.parametrize("kind", R.KINDS)
def test_gradient_against_differences(zf, kind):
    """L = sum(dy * norm(x)): its change along random directions of x, w and b, by central differences in 64 bits."""
    g = R.generator(77)
    rows, cols = 6, 48
    x, dy, w, b = R.normal(g, rows, cols), R.normal(g, rows, cols), R.normal(g, cols), R.normal(g, cols)
    mean, rstd = torch.empty(rows, device="cuda") if kind == "layer" else None, torch.empty(rows, device="cuda")
    k = zf.NORM_LAYER if kind == "layer" else zf.NORM_RMS
    zf.layer_norm(k, x, w, b, EPS, torch.empty_like(x), mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    zf.layer_norm_grad(k, dy, x, w, mean, rstd, dx, dw, db, R.bytes_buffer(zf.layer_norm_grad_bytes(rows, cols)))

    def loss(x, w, b):
        m = x.mean(1, keepdim=True) if kind == "layer" else 0.0
        return (dy.double() * ((x - m) / ((x - m).square().mean(1, keepdim=True) + EPS).sqrt() * w + b)).sum()
    at = [t.double() for t in (x, w, b)]
    for i, grad in enumerate((dx, dw, db)):
        to = R.normal(g, *at[i].shape).double()
        h = 1e-4
        plus, minus = ([t + s * h * to if j == i else t for j, t in enumerate(at)] for s in (1, -1))
        change = float((loss(*plus) - loss(*minus)) / (2 * h))
        # truncation h^2 / 6 of the third derivative (of order |dy| |to|^3 rstd^3 a row) and about 100 roundings of
        # binary32 against the terms' magnitudes
        room = float((grad.double() * to).abs().sum()) * 100 * R.U32 + h * h * 100 * rows * cols
        assert abs(float((grad.double() * to).sum()) - change) <= room
