"""Batches of many lengths with one workspace, made for the longest and with guards at its ends."""
import pytest
import torch

from tests import rank_ops as R
from tests import weight_grad_plan as plan

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


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


def whole(g, rows, cols):
    return torch.randint(-8, 9, (rows, cols), generator=g, device="cuda").to(BF16)


def test_table_gradients(zf):
    """At 2048 columns 8191 tokens take spans of 8, and twice the partial sums of 8192."""
    g, vocab, cols, longest = R.generator(1), 300, 2048, 8200
    d, ids = whole(g, longest, cols), torch.randint(-1, vocab, (longest,), generator=g, device="cuda")
    ws = R.bytes_buffer(zf.embedding_grad_bytes(longest, vocab, cols))
    for n in (8200, 8192, 8191, 8185, 4097, 4096, 100, 1):
        grad = torch.empty(vocab, cols, device="cuda")
        zf.embedding_grad(d[:n], ids[:n], grad, ws)
        at = torch.where(ids[:n] >= 0, ids[:n], vocab)
        want = torch.zeros(vocab + 1, cols, dtype=torch.float64, device="cuda").index_add_(0, at, d[:n].double())
        assert torch.equal(grad.double(), want[:-1]), n


@pytest.mark.parametrize("outs,ins,batches", [(256, 1024, (11300, 11264, 11263, 5000, 2047, 300, 1)),
                                              (1024, 1024, (8192, 8191, 4000, 1000, 31))])
def test_weight_gradients(zf, outs, ins, batches):
    g = R.generator(2)
    dy, x = whole(g, batches[0], outs), whole(g, batches[0], ins)
    codes, scales = R.keep(x)
    ws = R.bytes_buffer(zf.weight_grad_bytes(batches[0], outs, ins))
    for rows in batches:
        grad = torch.empty(outs, ins, device="cuda")
        zf.weight_grad(dy[:rows], zf.act8(codes[:rows], scales[:rows]), grad, ws)
        assert torch.equal(grad.double(), dy[:rows].double().t().contiguous() @ x[:rows].double()), rows


def test_a_weight_gradient_without_splits_takes_no_workspace(zf):
    """512 tokens of 2048 x 1536 are not split, though the size asked for is that of smaller tiles with two splits."""
    rows, outs, ins = 512, 2048, 1536
    assert plan.chosen(rows, outs, ins)[1] == 1
    g = R.generator(3)
    dy, x = whole(g, rows, outs), whole(g, rows, ins)
    grad = torch.empty(outs, ins, device="cuda")
    zf.weight_grad(dy, zf.act8(*R.keep(x)), grad, None)
    assert torch.equal(grad.double(), dy.double().t().contiguous() @ x.double())
