"""Muon steps of plans that differ in what else is in them, against the plain
form in 64 bits.  Tolerances in |error|_F, of the update for the iteration
(tests/test_gpu_muon.py), of the weights for the four binary32 roundings of
W dec - rate O."""
import math

import pytest
import torch

from fsdp_sharded_mixed_amd import workloads as W
from tests import gpu_common as G
from tests.test_gpu_muon import TOL, Model, plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    from fsdp_sharded_mixed_amd import zf as Z
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return Z


def matrices(*shapes):
    return [(r * c, 0, 0, r) for r, c in shapes]


def check_step(zf, m, products, rule="rows", lr=0.5):
    """One step without decay, clipping or Nesterov's term; products[i]: those
    of m's i-th matrix."""
    before = m.buffers()
    mhp = zf.muon_hparams(lr, momentum=0.9, weight_decay=0.0, nesterov=False,
                          scale_rule=zf.MUON_SCALE_RMS if rule == "rms" else zf.MUON_SCALE_ROWS)
    m.step(zf.hparams(1e-3, max_norm=0.0), mhp)
    for (at, r, c), n in zip(m.places(), products):
        p = slice(at, at + r * c)
        o = plain(m.momentum[p].view(r, c)).reshape(-1)
        rate = lr * (0.2 * math.sqrt(max(r, c)) if rule == "rms" else math.sqrt(max(1.0, r / c)))
        want = before["master"][p].double() - rate * o
        err = (m.master[p].double() - want).norm().item()
        size = (rate * o).norm().item()
        G.say(f"{r}x{c} products={n}: {err / size:.2e}")
        assert err <= TOL[n] * size + 4 * 2.0 ** -24 * (want.norm().item() + size), (r, c)


@pytest.mark.parametrize("rule", ["rows", "rms"])
def test_thin_matrices_beside_large_ones(zf, rule):
    """A thin matrix is as exact beside a layer as it is alone."""
    segs = matrices((1100, 1300), (1293, 4), (9, 1293), (40, 2000), (32, 900), (7, 5))
    m = Model(zf, segs, list(range(len(segs))), 2, W.PER_UNIT)
    check_step(zf, m, [1, 3, 3, 1, 3, 3], rule)


# What the launches choose by their blocks (tiles of symmetric products / of
# applications, 64 x 64 tiles a block of the load takes):
LARGE = matrices((2048, 2048), (2048, 4100), (4099, 2000), (2048, 2048))     # 256 / 256, 4
ROUND = matrices((1024, 1024), (1000, 1032), (2048, 1024)) + [(3, 0, 2, 0)] \
    + matrices((1024, 1024), (1024, 1024))                                   # 64 / 128, 1
TABLE = matrices(*[(1024, 2048), (1000, 2100), (2052, 1004), (1021, 2049), (2049, 1021)]) \
    + [(5, 0, 2, 0)] \
    + matrices(*[(1024, 2048), (1000, 2100), (2052, 1004), (1021, 2049), (2049, 1021)])
#                                             128 / 128, 4, and more matrices than arguments hold


def spread(err, size, r, c, limit, room):
    """No element, row or column far worse than the whole: err, r x c, of a
    matrix of norm `size` whose elements are alike, each held to the relative
    error `limit` and `room` besides.  Over 2^24 elements a normal deviate
    stays below 6 of its own deviations; a row of c has 1 + 5 / sqrt(c) times
    its mean norm at most."""
    one = size / math.sqrt(r * c)
    assert err.abs().max().item() <= 8 * limit * one + room
    for sums, n in ((err.square().sum(1), c), (err.square().sum(0), r)):
        worst = sums.max().sqrt().item()
        assert worst <= (1 + 5 / math.sqrt(n)) * limit * one * math.sqrt(n) + room * math.sqrt(n)


@pytest.mark.parametrize("segs,n,layout,gdt,pdt,nesterov,rule,reduced", [
    (LARGE, 2, W.GLOBAL_FLAT, "bf16", "bf16", True, "rms", False),
    (LARGE, 3, W.PER_PARAM_DIM0, "f16", None, False, "rows", False),
    (ROUND, 2, W.GLOBAL_FLAT, "bf16", "f16", True, "rows", False),
    (ROUND, 5, W.PER_UNIT, "bf16", None, True, "rms", True),
    (TABLE, 1, W.GLOBAL_FLAT, "f16", "f16", False, "rms", False),
    (TABLE, 2, W.PER_PARAM_DIM0, "bf16", "bf16", True, "rows", True)])
def test_steps_of_large_plans(zf, segs, n, layout, gdt, pdt, nesterov, rule, reduced):
    chosen = [i for i, s in enumerate(segs) if s[3] > 0]
    m = Model(zf, segs, chosen, n, layout, gdt=gdt, pdt=pdt, reduced=reduced)
    lr, mu, decay = 0.5, 0.9, 0.1
    before = m.buffers()
    mhp = zf.muon_hparams(lr, momentum=mu, weight_decay=decay, nesterov=nesterov,
                          scale_rule=zf.MUON_SCALE_RMS if rule == "rms" else zf.MUON_SCALE_ROWS)
    m.step(zf.hparams(1e-3, max_norm=0.05), mhp)
    gs = torch.tensor(zf.read_result(m.state).gs, device="cuda")
    total = m.shards
    if total is None:
        total = m.grads[0].float()
        for q in m.grads[1:]:
            total = total + q.float()
    g = total * gs
    moment = torch.tensor(mu, device="cuda") * before["momentum"] + g
    u = g + torch.tensor(mu, device="cuda") * moment if nesterov else moment
    for at, r, c in m.places():
        p = slice(at, at + r * c)
        assert torch.equal(m.momentum[p], moment[p])
        assert torch.equal(m.square[p], before["square"][p])
        if pdt:
            assert torch.equal(m.params[p], m.master[p].to(m.params.dtype))
        o = plain(u[p].view(r, c))
        rate = lr * (0.2 * math.sqrt(max(r, c)) if rule == "rms" else math.sqrt(max(1.0, r / c)))
        want = before["master"][p].view(r, c).double() * (1 - lr * decay) - rate * o
        err = m.master[p].view(r, c).double() - want
        size = (rate * o).norm().item()
        G.say(f"{r}x{c}: {err.norm().item() / size:.2e}")
        # four roundings of 2^-24 (the factor, two products, the difference)
        four = 4 * 2.0 ** -24
        assert err.norm().item() <= TOL[1] * size + four * (want.norm().item() + size)
        largest = want.abs().max().item() + (rate * o).abs().max().item()
        spread(err, size, r, c, TOL[1], four * largest)


@pytest.mark.parametrize("segs", [LARGE, ROUND, TABLE, matrices((4096, 4096)), matrices((4000, 4500))])
@pytest.mark.parametrize("products", [1, 3])
def test_large_batches(zf, segs, products):
    """The same tiles, and short sides above 2048, for either number of
    products."""
    from tests.test_gpu_muon import matrix, run
    shapes = [(s[3], s[0] // s[3]) for s in segs if s[3] > 0]
    xs = [matrix(r, c, torch.bfloat16, i) for i, (r, c) in enumerate(shapes)]
    ys = run(zf, xs, [torch.empty_like(x, dtype=torch.float32) for x in xs],
             zf.ns_params(products=products))
    for x, y in zip(xs, ys):
        want = plain(x)
        err, size = y.double() - want, want.norm().item()
        G.say(f"{tuple(x.shape)} products={products}: {err.norm().item() / size:.2e}")
        assert err.norm().item() <= TOL[products] * size
        spread(err, size, *x.shape, TOL[products], 0.0)


def test_matrices_in_shared_memory_take_three_products(zf):
    segs = matrices((128, 128), (16, 34), (96, 160), (64, 300), (300, 64), (96, 250), (1, 21), (33, 1))
    check_step(zf, Model(zf, segs, list(range(len(segs))), 2, W.GLOBAL_FLAT), [3] * len(segs))


def test_more_ranges_than_a_launch_takes(zf):
    """70 matrices with vectors of odd lengths between them: AdamW's part bit
    for bit as in zf_shard_step, over 71 ranges."""
    segs, chosen = [], []
    for i in range(70):
        segs.append((1 + i * 7 % 90, 0, 1, 0))
        chosen.append(len(segs))
        segs.append(((5 + i) * 9, 0, 0, 5 + i))
    segs.append((1000, 0, 1, 0))
    a, b = (Model(zf, segs, chosen, 3, W.GLOBAL_FLAT) for _ in range(2))
    hp = zf.hparams(2e-3, weight_decay=0.01, max_norm=0.05)
    a.step(hp, zf.muon_hparams(1e-2))
    b.adamw(hp)
    rest = torch.ones_like(a.real)
    for at, r, c in a.places():
        rest[at:at + r * c] = False
    for name in ("master", "momentum", "square", "params"):
        x, y = getattr(a, name), getattr(b, name)
        assert torch.equal(G.bits_view(x[rest]), G.bits_view(y[rest])), name
    assert not torch.equal(a.master[~rest], b.master[~rest])


@pytest.mark.parametrize("shape", [(1, 5), (5, 1), (24, 40), (300, 200), (5, 3000), (1100, 2048)])
@pytest.mark.parametrize("products", [1, 3])
@pytest.mark.parametrize("value", ["inf", "-inf", "nan"])
def test_one_element_without_a_value(zf, shape, products, value):
    """NaN throughout that matrix, the others as they are without it."""
    from tests.test_gpu_muon import matrix, run
    ns = zf.ns_params(products=products)
    xs = [matrix(*shape, torch.float32, i) for i in range(3)]
    clean = run(zf, xs, [torch.empty_like(x) for x in xs], ns)
    xs[1][shape[0] // 2, shape[1] - 1] = float(value)
    ys = run(zf, xs, [torch.empty_like(x) for x in xs], ns)
    assert torch.isnan(ys[1]).all()
    for k in (0, 2):
        assert torch.equal(G.bits_view(ys[k]), G.bits_view(clean[k]))


@pytest.mark.parametrize("segs", [TABLE, matrices(*[(40 + i, 90 - i) for i in range(20)])
                                  + [(7, 0, 2, 0)] + matrices((130, 1000), (20, 3000))])
def test_tables_captured_and_replayed(zf, segs):
    """Plans whose matrices travel through a table in the workspace: replays
    beside an eager twin, with new gradients between."""
    chosen = [i for i, s in enumerate(segs) if s[3] > 0]
    a, b = (Model(zf, segs, chosen, 2, W.GLOBAL_FLAT) for _ in range(2))
    hp, mhp = zf.hparams(1e-3), zf.muon_hparams(1e-2)
    for m in (a, b):
        m.step(hp, mhp)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(hp, mhp)
    g = torch.Generator(device="cuda").manual_seed(5)
    for k in range(3):
        for q, r in zip(a.grads, b.grads):
            q.copy_((torch.randn(q.shape, generator=g, device="cuda") * a.real).to(q.dtype))
            r.copy_(q)
        a.workspace.fill_(0xFF)
        graph.replay()
        b.step(hp, mhp)
        torch.cuda.synchronize()
        x, y = a.buffers(), b.buffers()
        for name in x:
            assert torch.equal(x[name].view(torch.uint8), y[name].view(torch.uint8)), (k, name)


def test_phase_events(zf):
    """Recorded in order around the passes."""
    m = Model(zf, ROUND, [0, 1, 2], 2, W.GLOBAL_FLAT)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    for e in events:
        e.record()  # makes the handle
    args = (m.muon, zf.hparams(1e-3), zf.muon_hparams(1e-2), *m.codes(), m.grads, m.master,
            m.momentum, m.square, m.params, m.workspace, m.state)
    for _ in range(2):
        zf.muon_step(*args, phase_events=[e.cuda_event for e in events])
        torch.cuda.synchronize()
        spans = [x.elapsed_time(y) for x, y in zip(events, events[1:])]
        assert all(s >= 0 for s in spans) and spans[2] > 0


def test_a_matrix_without_momentum_only_decays(zf):
    """Zero gradients on zero momentum: the update is zero."""
    segs = matrices((30, 40), (300, 500), (9, 2000), (1100, 1300))
    m = Model(zf, segs, [0, 1, 2, 3], 2, W.GLOBAL_FLAT)
    for t in m.grads + [m.momentum]:
        t.zero_()
    before = m.master.clone()
    m.step(zf.hparams(1e-3), zf.muon_hparams(0.25, weight_decay=0.5))
    assert torch.equal(m.master[m.real], (before * 0.875)[m.real])


@pytest.mark.parametrize("products", [1, 3])
@pytest.mark.parametrize("shape", [(40, 60), (500, 700), (1100, 1300)])
@pytest.mark.parametrize("norm", [1e-9, 1e-12, 1e-15, 1e-20])
def test_norms_far_below_eps(zf, shape, products, norm):
    """The result is a^5 X0 or so, which may be below what the operands hold:
    elements of X are rounded to 2^-46 (2^-25 of lo's scale of 2^21) at worst,
    in each of five steps, and grow."""
    from tests.test_gpu_muon import matrix, run
    x = matrix(*shape, torch.float32, 4)
    x *= norm / x.norm()
    y = run(zf, [x], [torch.empty_like(x)], zf.ns_params(products=products))[0]
    want = plain(x)
    least = 1.41 * 3.4445 ** 5 * 2.0 ** -46 * math.sqrt(x.numel())
    limit = 2.0 ** -8 if products == 1 else 2e-5
    assert (y.double() - want).norm().item() <= limit * want.norm().item() + least


@pytest.mark.parametrize("steps,coefficients", [
    (1, (3.4445, -4.7750, 2.0315)), (2, (3.4445, -4.7750, 2.0315)), (3, (3.4445, -4.7750, 2.0315)),
    (4, (3.4445, -4.7750, 2.0315)), (8, (3.4445, -4.7750, 2.0315)), (12, (1.5, -0.5, 0.0)),
    (6, (1.875, -1.25, 0.375))])
@pytest.mark.parametrize("shape", [(100, 140), (192, 320), (20, 2000), (1024, 1500)])
def test_other_iterations_with_one_product(zf, steps, coefficients, shape):
    from tests.test_gpu_muon import matrix, run
    a, b, c = coefficients
    x = matrix(*shape, torch.float32, 8)
    y = run(zf, [x], [torch.empty_like(x)],
            zf.ns_params(steps=steps, products=1, a=a, b=b, c=c))[0]
    want = plain(x, steps, coefficients=coefficients)
    err = (y.double() - want).norm().item() / want.norm().item()
    G.say(f"{shape} {steps} {coefficients}: {err:.2e}")
    assert err <= TOL[1]
