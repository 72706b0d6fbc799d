"""A rank's forward and backward calls as a program uses them: together on a plan's flat buffers up to the step,
captured in graphs, on several streams, and at offsets past 32 bits."""
import pytest
import torch

from tests import rank_ops as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


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


class Block:
    """A small model over a plan's flat buffers: embedding, RMS norm, one Linear.  Parameters are read from `flat`
    (16-bit, or the fp32 master), gradients added to each replica's fp32 main gradient."""
    vocab, hidden, outs, tokens, ranks = 97, 72, 56, 333, 3

    def __init__(self, zf, layout, flat_dtype):
        self.zf = zf
        sizes = [(self.vocab * self.hidden, 0, 0, self.vocab), (self.hidden, 1, 2, 0),
                 (self.outs * self.hidden, 1, 0, self.outs)]
        self.plan = zf.plan_flat(sizes, self.ranks, layout, 2)
        g = R.generator(layout + 17)
        self.size = self.plan.psi_pad
        # a parameter's first element: in the global flat one follows the other, under per-parameter shards each is a
        # unit, under per-unit plans the norm's weight and the Linear's lie in one
        at, self.at = 0, []
        for i, (n, unit, _, _) in enumerate(sizes):
            if layout == zf.GLOBAL_FLAT:
                self.at.append(at)
                at += n
            elif layout == zf.PER_PARAM_DIM0:
                self.at.append(self.plan.units[i].O)
            else:
                self.at.append(self.plan.units[unit].O + (self.hidden if i == 2 else 0))
        self.sizes = [s[0] for s in sizes]
        self.master = torch.zeros(self.size, device="cuda")
        for at, n in zip(self.at, self.sizes):
            self.master[at:at + n] = R.normal(g, n) * 0.1 + (1.0 if n == self.hidden else 0.0)
        self.flat = self.master.to(flat_dtype) if flat_dtype != F32 else self.master
        self.main = [torch.zeros(self.size, device="cuda") for _ in range(self.ranks)]
        self.ids = [torch.randint(-1, self.vocab, (self.tokens,), generator=g, device="cuda") for _ in self.main]
        self.dout = [R.normal(g, self.tokens, self.outs).to(BF16) for _ in self.main]
        t, h, o = self.tokens, self.hidden, self.outs
        self.x, self.y = (torch.empty(t, h, dtype=BF16, device="cuda") for _ in range(2))
        self.dx, self.dy = (torch.empty(t, h, dtype=BF16, device="cuda") for _ in range(2))
        self.rstd = torch.empty(t, device="cuda")
        self.x8, self.y8 = R.blank(zf, t, h), R.blank(zf, t, h)
        need = max(zf.embedding_grad_bytes(t, self.vocab, h), zf.layer_norm_grad_bytes(t, h),
                   zf.weight_grad_bytes(t, o, h))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")

    def part(self, buffer, i, *shape):
        return buffer[self.at[i]:self.at[i] + self.sizes[i]].view(*shape)

    def run(self, q, accumulate=True):
        """One replica's micro-batch: gradients of all three parameters."""
        zf, ws = self.zf, self.workspace
        zf.embedding(self.part(self.flat, 0, self.vocab, self.hidden), self.ids[q], self.x, scale=8.0)
        zf.layer_norm(zf.NORM_RMS, self.x, self.part(self.flat, 1, -1), None, EPS, self.y, None, self.rstd,
                      x8=self.x8, y8=self.y8)
        w = self.part(self.flat, 2, self.outs, self.hidden)
        self.dy.copy_(self.dout[q].float() @ w.float())  # the Linear's own products are a library's
        zf.weight_grad(self.dout[q], self.y8, self.part(self.main[q], 2, self.outs, self.hidden), ws, accumulate)
        zf.layer_norm_grad(zf.NORM_RMS, self.dy, self.x8, self.part(self.flat, 1, -1), None, self.rstd, self.dx,
                           self.part(self.main[q], 1, -1), None, ws, accumulate)
        zf.embedding_grad(self.dx, self.ids[q], self.part(self.main[q], 0, self.vocab, self.hidden), ws, 8.0,
                          accumulate)

    def wanted(self, q):
        """The gradients by the formulas in 64 bits, with the roundings that the types ask for, and bounds."""
        f, ids = self.flat.double(), self.ids[q]
        table, weight = self.part(f, 0, self.vocab, self.hidden), self.part(f, 1, -1)
        w = self.part(f, 2, self.outs, self.hidden)
        x = (torch.where((ids >= 0)[:, None], table[ids.clamp(min=0)], 0.0) * 8.0).to(BF16)
        x8 = R.numbers(*R.keep(x))
        r = (x.double().square().mean(1, keepdim=True) + EPS).rsqrt()
        y8 = R.numbers(*R.keep(self.y))  # y is compared by its own test; a code near a border may go either way
        dy = (self.dout[q].float() @ w.float()).to(BF16).double()
        xh, h = x8 * r, dy * weight
        dx = r * (h - xh * (h * xh).mean(1, keepdim=True))
        dw = (dy * xh).sum(0)
        table_grad = torch.zeros(self.vocab, self.hidden, dtype=torch.float64, device="cuda")
        table_size = torch.zeros_like(table_grad)
        real = ids >= 0
        table_grad.index_add_(0, ids[real], dx[real] * 8.0)
        table_size.index_add_(0, ids[real], dx[real].abs() * 8.0)
        linear = self.dout[q].double().t().contiguous() @ y8
        linear_size = self.dout[q].double().abs().t().contiguous() @ y8.abs()
        n, u = self.tokens, R.U32
        # rstd and dx carry about 100 roundings of binary32 at most, dx one of bf16
        return [(table_grad, table_size * (R.half_step(BF16) + (n + 300) * u) + 8 * n * R.least(BF16)),
                (dw, (dy * xh).abs().sum(0) * (n + 300) * u), (linear, linear_size * (n + 8) * 2 * u)]


@pytest.mark.parametrize("layout", [0, 1, 2])
@pytest.mark.parametrize("flat", [BF16, F32])
def test_gradients_into_the_step(zf, layout, flat):
    """Two micro-batches of three replicas: their main gradients are the formulas', the buckets' sums those of the
    replicas, and the step takes them."""
    b = Block(zf, layout, flat)
    want = []
    for q in range(b.ranks):
        b.run(q)
        b.run(q)
        want.append(b.wanted(q))
        for i, (total, error) in enumerate(want[-1]):
            got = b.part(b.main[q], i, *total.shape)
            R.assert_within(got, 2 * total, 2 * error + (2 * total.abs() + 2 * error) * R.U32, f"parameter {i}")
        real = torch.zeros(b.size, dtype=torch.bool, device="cuda")
        for at, n in zip(b.at, b.sizes):
            real[at:at + n] = True
        assert bool((b.main[q][~real] == 0).all()), "padding stays zero"
    shards = torch.empty(b.size, device="cuda")
    for group in range(b.plan.summary.n_groups):
        zf.bucket_reduce_scatter(b.plan, group, zf.F32, b.main, shards, False)
    total = b.main[0] + b.main[1] + b.main[2]
    assert torch.equal(shards, total)
    state = torch.empty(zf.state_bytes(), dtype=torch.uint8, device="cuda")
    zf.state_init(state, 1.0, False)
    m, v = torch.zeros_like(shards), torch.zeros_like(shards)
    ws = torch.empty(max(1, zf.workspace_bytes(b.plan)), dtype=torch.uint8, device="cuda")
    before = b.master.clone()

    def step():
        zf.shard_step(b.plan, zf.hparams(1e-2), zf.BF16, zf.BF16, None, b.master, m, v, None, ws, state,
                      grad_shards=shards, grads_reduced=True)
        return zf.read_result(state)
    result = step()
    assert result.skipped == 0 and result.t == 1
    assert abs(result.norm - float(total.double().norm()) / 3) <= 1e-5 * result.norm
    moved = before != b.master
    assert bool(moved[shards != 0].all())
    # a gradient that is not finite reaches the step's overflow check through any of the three
    for q in range(b.ranks):
        b.main[q].zero_()
    b.dout[1][5, 3] = float("nan")
    b.run(1)
    for group in range(b.plan.summary.n_groups):
        zf.bucket_reduce_scatter(b.plan, group, zf.F32, b.main, shards, False)
    kept = b.master.clone()
    assert step().skipped == 1 and torch.equal(b.master, kept)


def test_a_graph_replays_as_the_eager_calls(zf):
    """All calls of a micro-batch captured once; replays add to the main gradients with eager work between them, and
    with other tokens and gradients in the same buffers."""
    a, b = Block(zf, 1, BF16), Block(zf, 1, BF16)
    a.run(0)
    b.run(0)  # both warm
    for t in (a, b):
        for m in t.main:
            m.zero_()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        a.workspace.fill_(0xEE)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            a.run(0)
    torch.cuda.synchronize()
    g = R.generator(50)
    for k in range(5):
        ids = torch.randint(-1, a.vocab, (a.tokens,), generator=g, device="cuda")
        dout = R.normal(g, a.tokens, a.outs).to(BF16)
        for t in (a, b):
            t.ids[0].copy_(ids)
            t.dout[0].copy_(dout)
        a.workspace.fill_(k * 37)
        graph.replay()
        b.run(0)
        torch.cuda.synchronize()
        assert torch.equal(a.main[0], b.main[0]), f"replay {k}"
        for name in ("x", "y", "dx", "rstd"):
            assert torch.equal(getattr(a, name), getattr(b, name)), f"replay {k}: {name}"
        assert torch.equal(a.y8.codes, b.y8.codes) and torch.equal(a.x8.scales, b.x8.scales)


@pytest.mark.parametrize("tokens,vocab,cols", [(5000, 300, 64), (20000, 40960, 40), (100, 7, 24)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_a_graph_of_the_table_gradient(zf, tokens, vocab, cols, accumulate):
    """Each size of the sort, stored and added: counters and lists start anew in every replay."""
    g = R.generator(tokens)
    dout, ids = R.normal(g, tokens, cols).to(BF16), torch.zeros(tokens, dtype=torch.int64, device="cuda")
    grads = [torch.zeros(vocab, cols, device="cuda") for _ in range(2)]
    ws = [torch.empty(zf.embedding_grad_bytes(tokens, vocab, cols), dtype=torch.uint8, device="cuda") for _ in range(2)]
    zf.embedding_grad(dout, ids, grads[0], ws[0], 1.0, accumulate)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        zf.embedding_grad(dout, ids, grads[0], ws[0], 1.0, accumulate)
    grads[0].zero_()
    for k in range(4):
        ids.copy_(torch.randint(-2, vocab if k % 2 else min(vocab, 3), (tokens,), generator=g, device="cuda"))
        graph.replay()
        zf.embedding_grad(dout, ids, grads[1], ws[1], 1.0, accumulate)
        torch.cuda.synchronize()
        assert torch.equal(grads[0], grads[1]), f"replay {k}"


def test_two_streams(zf):
    """Calls on two streams at once, each with buffers and a workspace of its own."""
    blocks = [Block(zf, 1, BF16) for _ in range(3)]
    blocks[0].run(0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, b in zip(streams, blocks[1:]):
            with torch.cuda.stream(s):
                b.run(0, accumulate=False)
    torch.cuda.synchronize()
    for b in blocks[1:]:
        assert torch.equal(b.main[0], blocks[0].main[0])
    s = streams[0]  # the stream given, not the current one
    out = torch.empty_like(blocks[0].x)
    b = blocks[0]
    zf.embedding(b.part(b.flat, 0, b.vocab, b.hidden), b.ids[0], out, scale=8.0, stream=s)
    s.synchronize()
    assert torch.equal(out, b.x)


def free():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_norms_past_32_bits(zf):
    """More than 2^32 bytes and 2^31 elements: the last rows are as those of a small call."""
    rows, cols, last = (1 << 21) + 77, 1040, 500
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    x[:] = R.normal(R.generator(1), 1, cols).to(BF16)
    x[-last:] = R.normal(R.generator(2), last, cols).to(BF16)
    w = R.normal(R.generator(3), cols).to(BF16)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    a = zf.act8(torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                torch.empty(rows, -(-cols // 32), dtype=torch.uint8, device="cuda"))
    zf.layer_norm(zf.NORM_LAYER, x, w, w, EPS, y, mean, rstd, x8=a)
    tail = x[-last:].clone()
    y2, m2, r2 = torch.empty_like(tail), torch.empty(last, device="cuda"), torch.empty(last, device="cuda")
    zf.layer_norm(zf.NORM_LAYER, tail, w, w, EPS, y2, m2, r2)
    assert torch.equal(y[-last:], y2) and torch.equal(mean[-last:], m2) and torch.equal(rstd[-last:], r2)
    codes, scales = R.keep(tail)
    assert torch.equal(a.codes[-last:], codes) and torch.equal(a.scales[-last:], scales)
    dx = x  # x is not needed any more; dy is y
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(zf.layer_norm_grad_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    zf.layer_norm_grad(zf.NORM_LAYER, y, a, w, mean, rstd, dx, dw, db, ws)
    d2 = torch.empty_like(tail)
    zf.layer_norm_grad(zf.NORM_LAYER, y2, R.kept(zf, tail), w, m2, r2, d2, None, None, None)
    assert torch.equal(dx[-last:], d2)
    total, size = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2))
    for part in y.split(1 << 18):
        total += part.double().sum(0)
        size += part.double().abs().sum(0)
    # a sum of n terms takes n - 1 additions, each off by U32 of at most the sum of magnitudes
    R.assert_within(db, total, rows * R.U32 * size, "db")
    del x, y, a, dx
    free()


def test_tables_past_32_bits(zf):
    """A table and its gradient of more than 2^32 bytes: rows at its end."""
    vocab, cols, n = (1 << 20) + 33, 1032, 700
    table = torch.zeros(vocab, cols, device="cuda")
    table[-100:] = R.normal(R.generator(1), 100, cols)
    ids = vocab - 1 - torch.randint(0, 120, (n,), generator=R.generator(2), device="cuda")
    ids[::50] = 0
    out = torch.empty(n, cols, device="cuda")
    zf.embedding(table, ids, out)
    assert torch.equal(out, table[ids])
    grad = table.fill_(3.0)
    ws = torch.empty(zf.embedding_grad_bytes(n, vocab, cols), dtype=torch.uint8, device="cuda")
    zf.embedding_grad(out, ids, grad, ws)
    want = torch.zeros(vocab - int(ids[ids > 0].min()), cols, dtype=torch.float64, device="cuda")
    first, far = vocab - len(want), ids > 0
    size = torch.zeros_like(want)
    want.index_add_(0, ids[far] - first, out[far].double())
    size.index_add_(0, ids[far] - first, out[far].double().abs())
    R.assert_within(grad[first:], want, size * n * R.U32 + R.least(F32), "grad")
    assert bool((grad[1:first] == 0).all())
    del table, grad
    free()


def test_weight_gradients_past_32_bits(zf):
    """More than 2^32 bytes of upstream gradients: whole numbers, so that the product is exact."""
    rows, outs, ins = (1 << 18) + 21, 8704, 64
    g = R.generator(3)
    dy = torch.randint(-1, 2, (rows, outs), generator=g, device="cuda", dtype=torch.int8).to(BF16)
    x = torch.randint(-1, 2, (rows, ins), generator=g, device="cuda").to(BF16)
    grad = torch.empty(outs, ins, device="cuda")
    ws = torch.empty(max(1, zf.weight_grad_bytes(rows, outs, ins)), dtype=torch.uint8, device="cuda")
    zf.weight_grad(dy, R.kept(zf, x), grad, ws)
    want = torch.zeros(outs, ins, device="cuda")
    for a, b in zip(dy.split(1 << 15), x.split(1 << 15)):
        want += a.float().t().contiguous() @ b.float()
    assert torch.equal(grad, want)
    del dy, x
    free()
