"""The embedding lookup and its gradient against their definitions."""
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


def some_ids(g, n, vocab, dtype, kind):
    """kind: even; often (half of them one of three); one (all the same); none (all outside); each (in order, again
    and again)."""
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    if kind == "often":
        ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, ids % min(3, vocab), ids)
    elif kind == "one":
        ids = torch.full_like(ids, vocab - 1)
    elif kind == "none":
        ids = torch.where(ids % 2 == 0, -1 - ids, vocab + ids)
    elif kind == "each":
        ids = torch.arange(n, device="cuda") % vocab
    if kind in ("even", "often") and n > 2:
        outside = torch.rand(n, generator=g, device="cuda") < 0.1
        ids = torch.where(outside, torch.where(ids % 2 == 0, -1, vocab), ids)
    return ids.to(dtype)


def real(ids, vocab):
    return (ids >= 0) & (ids < vocab)


@pytest.mark.parametrize("table,out", [(BF16, BF16), (F32, BF16), (F16, F16), (F32, F32), (F16, F32), (F32, F16)])
@pytest.mark.parametrize("n,vocab,cols,gap,skew,scale", [
    (1, 1, 1, 0, 0, 1.0), (1, 7, 8, 0, 1, 32.0), (5, 3, 33, 2, 1, 0.5), (128, 1024, 1024, 0, 0, 32.0),
    (77, 50, 777, 1, 3, 1.7), (300, 999, 2048, 8, 0, 1.0), (9, 40, 5001, 0, 1, -2.0)])
def test_lookup(zf, table, out, n, vocab, cols, gap, skew, scale):
    g = R.generator(n + cols)
    t = R.filled(R.normal(g, vocab, cols), table, 0, skew, "table")
    ids = some_ids(g, n, vocab, torch.int64 if n % 2 else torch.int32, "even")
    got = R.buffer(n, cols, out, gap, skew, "out")
    zf.embedding(t, ids, got, scale=scale)
    scale32 = torch.tensor(scale, dtype=F32, device="cuda")
    rows = t[ids.long().clamp(0, vocab - 1)].float() * scale32  # one rounding of binary32, then one to the type
    assert torch.equal(got, torch.where(real(ids, vocab)[:, None], rows, 0.0).to(out))


def test_lookup_of_what_is_not_finite(zf):
    """Rows of infinities and NaN reach their own tokens only; padding stays zero."""
    t = torch.ones(4, 16, dtype=BF16, device="cuda")
    t[1], t[2] = float("inf"), float("nan")
    out = torch.empty(5, 16, dtype=BF16, device="cuda")
    zf.embedding(t, torch.tensor([0, 1, -1, 2, 1 << 40], device="cuda"), out, scale=2.0)
    assert bool((out[0] == 2).all() and out[1].isinf().all() and out[3].isnan().all())
    assert bool((out[[2, 4]] == 0).all())


def check_grad(zf, ids, dout, vocab, grad_dtype, accumulate, scale, skew=0):
    n, cols = dout.shape
    g = R.generator(5)
    grad = R.filled(R.normal(g, vocab, cols), grad_dtype, 0, skew, "grad")
    old = grad.clone()
    ws = R.bytes_buffer(max(1, zf.embedding_grad_bytes(n, vocab, cols)))
    zf.embedding_grad(dout, ids, grad, ws, scale=scale, accumulate=accumulate)
    fine = real(ids, vocab)
    at, rows = ids[fine].long(), dout[fine].double()
    total = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, at, rows)
    size = torch.zeros_like(total).index_add_(0, at, rows.abs())
    count = torch.bincount(at, minlength=vocab).double()[:, None] if len(at) else torch.zeros(vocab, 1, device="cuda")
    scale = float(torch.tensor(scale, dtype=F32))
    # a sum of m terms takes m - 1 additions, each off by U32 of what it holds, and the scale one more rounding
    error = abs(scale) * size * count * R.U32 * 1.001
    want, bound = R.written(total * scale, error, old, grad_dtype, accumulate)
    if accumulate:  # rows without tokens are not touched
        empty = count[:, 0] == 0
        assert torch.equal(grad[empty], old[empty])
    R.assert_within(grad, want, bound, "grad")
    return grad


@pytest.mark.parametrize("dout,grad", [(BF16, F32), (BF16, BF16), (F16, F16), (F32, F32)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab,cols,kind,gap,skew", [
    (1, 1, 1, "even", 0, 0), (1, 9, 8, "one", 0, 1), (2, 3, 17, "none", 1, 0), (7, 5, 33, "often", 0, 1),
    (64, 1, 64, "one", 0, 0), (100, 1000, 40, "even", 3, 3), (1000, 1024, 1024, "often", 0, 0),
    (1500, 777, 100, "one", 0, 0), (4096, 511, 72, "each", 0, 0), (4097, 512, 65, "often", 0, 1),
    (9000, 40960, 48, "even", 8, 0), (20000, 300, 16, "often", 0, 0), (513, 60, 4100, "often", 0, 0)])
def test_gradient(zf, dout, grad, accumulate, n, vocab, cols, kind, gap, skew):
    g = R.generator(n * 7 + cols)
    d = R.filled(R.normal(g, n, cols) * 0.1, dout, gap, skew, "dout")
    ids = some_ids(g, n, vocab, torch.int32 if n % 2 else torch.int64, kind)
    check_grad(zf, ids, d, vocab, grad, accumulate, 32.0 if cols == 1024 else 0.37, skew)


def test_one_token_that_fills_a_long_batch(zf):
    """A run over thousands of spans, and a batch that takes several blocks and three passes of the sort."""
    g = R.generator(3)
    d = (R.normal(g, 70001, 24) * 0.1).to(BF16)
    ids = torch.full((70001,), 300000, device="cuda")
    ids[::1000] = torch.randint(0, 300001, (71,), generator=g, device="cuda")
    check_grad(zf, ids, d, 300001, F32, False, 1.0)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["even", "often", "one", "none", "each", "runs"])
@pytest.mark.parametrize("n,cols", [(1, 512), (7, 520), (8, 512), (9, 2048), (17, 1024), (100, 512), (1000, 2056),
                                    (4096, 512), (4100, 1024), (8192, 2048), (9001, 2048), (12288, 2048), (16385, 2048)])
def test_whole_numbers_in_rows_of_whole_waves(zf, accumulate, kind, n, cols):
    """Small whole numbers, so that every sum is exact: the sums of runs that end anywhere in and behind their spans."""
    g = R.generator(n + cols)
    vocab = 700
    d = torch.randint(-8, 9, (n, cols), generator=g, device="cuda").to(BF16)
    if kind == "runs":  # run lengths 1, 2, .. 60, again and again, in a random order
        lengths = torch.arange(n, device="cuda") % 60 + 1
        ids = torch.arange(n, device="cuda").repeat_interleave(lengths)[:n] % vocab
        ids = ids[torch.randperm(n, generator=g, device="cuda")]
    else:
        ids = some_ids(g, n, vocab, torch.int64, kind)
    grad = torch.ones(vocab, cols, device="cuda")
    zf.embedding_grad(d, ids, grad, R.bytes_buffer(zf.embedding_grad_bytes(n, vocab, cols)), scale=2.0,
                      accumulate=accumulate)
    fine = real(ids, vocab)
    want = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, ids[fine].long(), d[fine].double())
    assert torch.equal(grad.double(), want * 2 + (1 if accumulate else 0))


@pytest.mark.parametrize("n", [5, 5000])
def test_a_vocabulary_of_many_rows(zf, n):
    """2^27 and more rows of one element: what clears the gradient looks after 2^18 of them at a time, and the sort
    takes four passes."""
    vocab = (1 << 27) + 5
    g = R.generator(n)
    grad = torch.ones(vocab, 1, dtype=BF16, device="cuda")
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    ids[0], ids[1] = vocab - 1, 0
    d = torch.randint(1, 9, (n, 1), generator=g, device="cuda").to(BF16)
    zf.embedding_grad(d, ids, grad, R.bytes_buffer(zf.embedding_grad_bytes(n, vocab, 1)))
    want = torch.zeros(vocab, device="cuda").index_add_(0, ids, d[:, 0].float())
    assert torch.equal(grad[:, 0], want.to(BF16))


def test_the_same_call_gives_the_same_bits(zf):
    g = R.generator(8)
    d = R.normal(g, 12345, 130).to(BF16)
    ids = some_ids(g, 12345, 500, torch.int64, "often")
    ws = R.bytes_buffer(zf.embedding_grad_bytes(12345, 500, 130))
    got = []
    for k in range(3):
        ws.fill_(0x11 * k)
        got.append(torch.empty(500, 130, device="cuda"))
        zf.embedding_grad(d, ids, got[-1], ws)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_no_tokens(zf):
    none, d = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 8, dtype=BF16, device="cuda")
    zf.embedding(torch.ones(3, 8, dtype=BF16, device="cuda"), none, d)
    grad = R.filled(torch.ones(3, 8, device="cuda"), F32)
    zf.embedding_grad(d, none, grad, None, accumulate=True)
    assert bool((grad == 1).all())
    zf.embedding_grad(d, none, grad, None, accumulate=False)
    assert bool((grad == 0).all())


def test_what_is_not_finite_stays_in_its_row(zf):
    """An infinity or a NaN in dout reaches its own row and column only, and padding's not at all."""
    d = torch.ones(6, 20, dtype=BF16, device="cuda")
    d[1, 3], d[4, 5], d[5] = float("inf"), float("nan"), float("nan")
    ids = torch.tensor([0, 1, 2, 1, 2, -1], device="cuda")
    grad = torch.full((4, 20), 9.0, device="cuda")
    zf.embedding_grad(d, ids, grad, R.bytes_buffer(zf.embedding_grad_bytes(6, 4, 20)))
    want = torch.tensor([1.0, 2.0, 2.0, 0.0], device="cuda")[:, None].repeat(1, 20)
    want[1, 3], want[2, 5] = float("inf"), float("nan")
    assert torch.equal(grad.isnan(), want.isnan())
    assert torch.equal(grad.nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))


def test_gradient_against_differences(zf):
    """The lookup is linear in the table: the loss's change along a direction is the gradient's product with it."""
    g = R.generator(12)
    table, direction = R.normal(g, 50, 64), R.normal(g, 50, 64)
    ids = some_ids(g, 200, 50, torch.int64, "often")
    d = R.normal(g, 200, 64)
    grad = torch.empty(50, 64, device="cuda")
    zf.embedding_grad(d, ids, grad, R.bytes_buffer(zf.embedding_grad_bytes(200, 50, 64)), scale=3.0)
    fine = real(ids, 50)

    def loss(t):
        return float((t.double()[ids[fine].long()] * 3.0 * d[fine].double()).sum())
    change = (loss(table.double() + direction.double()) - loss(table.double() - direction.double())) / 2
    terms = float((d[fine].double().abs() * 3.0 * direction.double().abs()[ids[fine].long()]).sum())
    assert abs(float((grad.double() * direction.double()).sum()) - change) <= terms * 200 * R.U32
