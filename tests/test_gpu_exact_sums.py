"""Sums over long batches in whole numbers: every partial sum is exact in binary32, whatever its order, so a row that is
left out or taken twice shows wherever it lies."""
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


def whole(g, most, rows, cols, dtype):
    return torch.randint(-most, most + 1, (rows, cols), generator=g, device="cuda", dtype=torch.int8).to(dtype)


def sums(parts, cols):
    """Sums of the columns of (dy, xh) and of dy, part by part in 64 bits."""
    dw, db = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2))
    for dy, xh in parts:
        dy = dy.double()
        dw += (dy * xh.double()).sum(0)
        db += dy.sum(0)
    return dw, db


# the last two give a block thousands of rows
@pytest.mark.parametrize("rows,cols,most", [(40000, 24, 4), (20000, 200, 4), (9000, 2100, 4), (9000, 2096, 4), (3001, 1000, 4),
                                            (700, 8200, 4), (1500, 17000, 4), (4000003, 24, 1), (4000003, 15, 1)])
@pytest.mark.parametrize("kind", R.KINDS)
@pytest.mark.parametrize("kept", [False, True])
def test_norm_gradients(zf, kind, kept, rows, cols, most):
    """rstd is a power of two and the mean a whole number (as a caller may give them), so xh is exact: |dy xh| is at most
    64 (one at a time in the longest batches), a column's sum below 2^24 halves."""
    g = R.generator(rows + cols)
    x, dy = whole(g, most, rows, cols, BF16), whole(g, most, rows, cols, BF16)
    rstd = torch.exp2(torch.randint(-1, 2 if most > 1 else 1, (rows,), generator=g, device="cuda").float())
    mean = torch.randint(-2, 3, (rows,), generator=g, device="cuda").float() if kind == "layer" else None
    if most == 1:
        mean = torch.zeros(rows, device="cuda") if kind == "layer" else None
    w = torch.ones(cols, dtype=BF16, device="cuda")
    dw, db = R.buffer(1, cols, F32, 0, 1).view(-1), R.buffer(1, cols, F32, 0, 1).view(-1)
    dw.fill_(3.0)
    db.fill_(-5.0)
    given = x
    if kept:
        given = zf.act8(torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                        torch.empty(rows, -(-cols // 32), dtype=torch.uint8, device="cuda"))
        zf.act8_store(given, x)
    ws = R.bytes_buffer(zf.layer_norm_grad_bytes(rows, cols))
    zf.layer_norm_grad(zf.NORM_LAYER if kind == "layer" else zf.NORM_RMS, dy, given, w, mean, rstd, torch.empty_like(dy),
                       dw, db, ws, accumulate=True)

    def parts():
        for at in range(0, rows, 1 << 18):
            s = slice(at, at + (1 << 18))
            yield dy[s], (x[s].float() - (mean[s, None] if kind == "layer" else 0.0)) * rstd[s, None]
    want_w, want_b = sums(parts(), cols)
    assert float(want_w.abs().max()) < 2 ** 23
    assert torch.equal(dw.double(), want_w + 3) and torch.equal(db.double(), want_b - 5)


def test_norm_gradients_past_32_bits(zf):
    """More than 2^31 elements: both columns' sums, exact."""
    rows, cols = (1 << 21) + 77, 1040
    g = R.generator(1)
    x, dy = whole(g, 1, rows, cols, BF16), whole(g, 1, rows, cols, BF16)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(zf.layer_norm_grad_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    want = sums(zip(dy.split(1 << 18), x.split(1 << 18)), cols)
    zf.layer_norm_grad(zf.NORM_LAYER, dy, x, torch.ones(cols, device="cuda"), mean, rstd, dy, dw, db, ws)
    assert torch.equal(dw.double(), want[0]) and torch.equal(db.double(), want[1])
    del x, dy
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def table_gradient(zf, ids, d, vocab, accumulate):
    grad = torch.ones(vocab, d.shape[1], device="cuda")
    ws = R.bytes_buffer(zf.embedding_grad_bytes(len(ids), vocab, d.shape[1]))
    zf.embedding_grad(d, ids, grad, ws, accumulate=accumulate)
    fine = (ids >= 0) & (ids < vocab)
    want = torch.full(grad.shape, 1.0 if accumulate else 0.0, dtype=torch.float64, device="cuda")
    want.index_add_(0, ids[fine].long(), d[fine].double())
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(grad.double(), want)


@pytest.mark.parametrize("cols", [24, 1024])
def test_one_token_that_fills_a_long_batch(zf, cols):
    """A run over thousands of spans beside single tokens, in rows of part of a wave and of two."""
    g = R.generator(3)
    ids = torch.full((70001,), 3000, device="cuda")
    ids[::1000] = torch.randint(0, 3001, (71,), generator=g, device="cuda")
    table_gradient(zf, ids, whole(g, 8, 70001, cols, BF16), 3001, False)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab", [((1 << 20) + 77, 300001), ((1 << 20) + 77, 500), ((1 << 21) + 1025, 40960)])
def test_tables_of_batches_past_a_sort_blocks_thousand(zf, n, vocab, accumulate):
    """Above 2^20 tokens a block of the sort takes 2048 tokens and more: one to three passes, half of the tokens one of
    three ids, a tenth outside."""
    g = R.generator(n + vocab)
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, ids % 3, ids)
    ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.1, -1, ids).to(torch.int32)
    table_gradient(zf, ids, whole(g, 4, n, 8, BF16), vocab, accumulate)
