"""Orthogonalisation and the Muon step on the GPU against plain 64-bit forms.

Tolerances, in |error|_F / |X|_F.  u is half a step of the operands: 2^-11
for one product, 2^-22 for three.  One iteration takes roundings of X (into
B X and, twice, into A), of A and of B, all off the diagonal.  With singular
values up to 1.2, |B|_2 and |A|_2's factor |b + 2 c A|_2 below 4.8, they give
in the worst case, all aligned, (3.5 + 2 + 4.8 * 3 * 1.2) u = 23 u; rounding
errors are spread evenly over +-u (0.58 u root mean square at most, 0.41 u on
average over a binade) and the last factor is near 0.7 where the singular
values end, so that about 3.4 u arises per iteration, and at most two
iterations' worth survives (the map's slope is below 1 over most of [0.3,
1.1], where the last iterations run): 7 u.  For one product that is 3.4e-3,
taken as 2^-8.  For three products the operands' part is 1.7e-6; the 32-bit
sums of up to 8192 terms add 2^-25 sqrt(8192) = 2.7e-6 per product, times
the same 3.4 * 2: 2e-5 covers both.  The destination's rounding adds
finfo(dtype).eps / 2.
"""
import math

import numpy as np
import pytest
import torch

from fsdp_sharded_mixed_amd import workloads as W
from tests import gpu_common as G

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
TOL = {1: 2.0 ** -8, 3: 2e-5}
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def zf():
    from fsdp_sharded_mixed_amd import zf as Z
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return Z


def plain(x, steps=5, eps=1e-7, coefficients=NS):
    """The iteration in 64 bits, on the device."""
    a, b, c = coefficients
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t().contiguous()
    x = x / (x.square().sum().sqrt() + eps)
    for _ in range(steps):
        g = x @ x.t().contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.t() if tall else x


def off(got, want):
    d = (got.double() - want).norm().item()
    n = want.norm().item()
    return d / n if n else d


def limit(products, dtype):
    return TOL[products] + torch.finfo(dtype).eps / 2


def matrix(rows, cols, dtype, seed, gap=0, kind="gauss"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    if kind == "rank":
        r = min(4, rows, cols)
        x = x * 0.1 + (torch.randn(rows, r, generator=g, device="cuda")
                       @ torch.randn(r, cols, generator=g, device="cuda"))
    if kind == "decay":  # singular values 1/i
        u, _, v = torch.linalg.svd(x.double(), full_matrices=False)
        s = 1.0 / torch.arange(1, u.shape[1] + 1, device="cuda", dtype=torch.float64)
        x = (u * s) @ v
    wide = torch.full((rows, cols + gap), 7.0, dtype=dtype, device="cuda")
    wide[:, :cols] = (x * 1e-2).to(dtype)
    return wide


def run(zf, mats, outs, ns=None, stream=None):
    b = zf.ortho_batch(mats, outs)
    ws = torch.empty(zf.orthogonalize_bytes(b, ns), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # NaN patterns: nothing may be read before it is written
    zf.orthogonalize(b, ws, ns=ns, stream=stream)
    torch.cuda.synchronize()
    return outs


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 2), (3, 64), (16, 34), (63, 65), (64, 64), (65, 64),
          (128, 40), (128, 128), (129, 257), (257, 1000), (1000, 333), (200, 4097), (1024, 1024),
          (5, 8191)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("src,dst", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"),
                                     ("f32", "f32")])
def test_orthogonalize(zf, rows, cols, src, dst):
    x = matrix(rows, cols, DT[src], 11)
    y = torch.empty(rows, cols, dtype=DT[dst], device="cuda")
    run(zf, [x], [y])
    err = off(y, plain(x))
    G.say(f"{rows}x{cols} {src}->{dst}: {err:.2e}")
    assert err <= limit(1 if dst == "bf16" else 3, DT[dst])


@pytest.mark.parametrize("kind", ["rank", "decay"])
@pytest.mark.parametrize("rows,cols", [(96, 160), (512, 512), (700, 300), (256, 2048)])
@pytest.mark.parametrize("products", [1, 3])
def test_spectra(zf, kind, rows, cols, products):
    x = matrix(rows, cols, torch.float32, 5, kind=kind)
    y = torch.empty(rows, cols, device="cuda")
    run(zf, [x], [y], zf.ns_params(products=products))
    err = off(y, plain(x))
    G.say(f"{kind} {rows}x{cols} products={products}: {err:.2e}")
    assert err <= limit(products, torch.float32)


@pytest.mark.parametrize("rows,cols", [(11, 2000), (64, 1400), (100, 1500), (1500, 100),
                                       (128, 8192), (300, 300), (2048, 2048)])
@pytest.mark.parametrize("count", [1, 24])
def test_few_strong_directions_over_noise(zf, rows, cols, count):
    """One matrix (single steps) and a batch of more than a round of blocks
    (steps in pairs where the matrices are long): singular values 30 apart,
    whose squares are what the products hold."""
    if rows * cols * count > 1 << 26:
        count = 4
    xs = []
    for seed in range(count):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = min(8, rows, cols)
        strong = (torch.randn(rows, r, generator=g, device="cuda")
                  @ torch.randn(r, cols, generator=g, device="cuda"))
        xs.append(torch.randn(rows, cols, generator=g, device="cuda") + strong * (2 / math.sqrt(r)))
    ys = run(zf, xs, [torch.empty_like(x) for x in xs], zf.ns_params(products=1))
    worst = max(off(y, plain(x)) for x, y in zip(xs, ys))
    G.say(f"{count} of {rows}x{cols}: {worst:.2e}")
    assert worst <= limit(1, torch.float32)


def test_batch_of_many_shapes_with_strides(zf):
    shapes = [(1, 77), (65, 1), (257, 300), (300, 257), (64, 64), (130, 1030), (999, 101)] * 4
    wide = [matrix(r, c, torch.float16, i, gap=3) for i, (r, c) in enumerate(shapes)]
    outs = [torch.full((r, c + 5), 3.0, dtype=torch.bfloat16, device="cuda") for r, c in shapes]
    run(zf, [w[:, :c] for w, (_, c) in zip(wide, shapes)],
        [o[:, :c] for o, (_, c) in zip(outs, shapes)])
    for w, o, (r, c) in zip(wide, outs, shapes):
        assert off(o[:, :c], plain(w[:, :c])) <= limit(1, torch.bfloat16)
        assert (o[:, c:] == 3.0).all() and (w[:, c:] == 7.0).all()


def test_the_same_call_gives_the_same_bits(zf):
    shapes = [(100, 200), (512, 256), (33, 33)]
    xs = [matrix(r, c, torch.float32, i) for i, (r, c) in enumerate(shapes)]
    together = run(zf, xs, [torch.empty_like(x, dtype=torch.bfloat16) for x in xs])
    again = run(zf, xs, [torch.empty_like(x, dtype=torch.bfloat16) for x in xs])
    for a, b in zip(together, again):
        assert torch.equal(G.bits_view(a), G.bits_view(b))


def test_more_matrices_than_a_launch_takes_as_arguments(zf):
    """70 matrices for the products and 20 held in shared memory, mixed: the
    tables of both, and the search through more first blocks than travel."""
    shapes = [(130 + i, 200 - i) for i in range(70)]
    for i in range(20):
        shapes.insert(4 * i, (5 + i, 90 - 3 * i))
    xs = [matrix(r, c, torch.float32, i) for i, (r, c) in enumerate(shapes)]
    ys = run(zf, xs, [torch.empty_like(x, dtype=torch.bfloat16) for x in xs])
    for x, y in zip(xs, ys):
        assert off(y, plain(x)) <= limit(1, torch.bfloat16), tuple(x.shape)


def test_longest_side_and_more_than_one_group(zf):
    """Five of 2^26 padded elements: the workspace holds four at a time.  (The
    sums have 2^20 terms: 2^-25 sqrt(2^20) = 3e-5, within the one product's
    tolerance.)"""
    shapes = [(60, 1 << 20), (1 << 20, 60), (33, (1 << 20) - 5), (7, 1 << 20), (64, 1 << 20)]
    xs = [matrix(r, c, torch.bfloat16, i) for i, (r, c) in enumerate(shapes)]
    one = zf.orthogonalize_bytes(zf.ortho_batch(xs[:4], [torch.empty_like(x) for x in xs[:4]]))
    b = zf.ortho_batch(xs, [torch.empty_like(x) for x in xs])
    assert zf.orthogonalize_bytes(b) < 1.01 * one
    ys = run(zf, xs, b.tensors[5:])
    for x, y in zip(xs, ys):
        assert off(y, plain(x)) <= limit(1, torch.bfloat16), tuple(x.shape)


def test_in_place(zf):
    x = matrix(130, 70, torch.float32, 3, gap=2)
    want = plain(x[:, :70])
    run(zf, [x[:, :70]], [x[:, :70]])
    assert off(x[:, :70], want) <= limit(3, torch.float32)
    assert (x[:, 70:] == 7.0).all()


@pytest.mark.parametrize("shape", [(40, 24), (24, 40), (300, 200), (1, 5)])
def test_zeros_and_nonfinite_matrices_stay_apart(zf, shape):
    xs = [matrix(*shape, torch.float32, i) for i in range(5)]
    xs[1].zero_()
    xs[2][-1, 0] = float("inf")
    xs[3][0, -1] = float("nan")
    clean = run(zf, [xs[0], xs[4]], [torch.empty_like(xs[0]) for _ in range(2)])
    ys = run(zf, xs, [torch.empty_like(x) for x in xs])
    assert torch.equal(ys[0], clean[0]) and torch.equal(ys[4], clean[1])
    assert (ys[1] == 0).all()
    if shape != (1, 5):
        assert torch.isnan(ys[2]).all()
        assert torch.isnan(ys[3]).all()
    assert not torch.isfinite(ys[2]).any() or shape == (1, 5)


@pytest.mark.parametrize("factor", [1e-30, 1e-42, 1e30, 3e38])
def test_extreme_magnitudes(zf, factor):
    # 32-bit squares would overflow or vanish: the norm is taken in 64 bits
    x = torch.randn(70, 50, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x = (x.clamp(-1, 1).double() * factor).float()
    y = torch.empty_like(x)
    run(zf, [x], [y], zf.ns_params(eps=0.0))
    assert off(y, plain(x, eps=0.0)) <= limit(3, torch.float32)


@pytest.mark.parametrize("steps,coefficients", [(1, NS), (2, NS), (12, (1.5, -0.5, 0.0)),
                                                (6, (1.875, -1.25, 0.375))])
def test_other_iterations(zf, steps, coefficients):
    x = matrix(192, 320, torch.float32, 8)
    y = torch.empty_like(x)
    a, b, c = coefficients
    run(zf, [x], [y], zf.ns_params(steps=steps, products=3, a=a, b=b, c=c))
    assert off(y, plain(x, steps, coefficients=coefficients)) <= limit(3, torch.float32)


def test_workspace_guards(zf):
    """The exact workspace between guard bands, and the outputs too."""
    shapes = [(257, 130), (64, 700), (3, 3)]
    xs = [matrix(r, c, torch.float32, i) for i, (r, c) in enumerate(shapes)]
    outs = [torch.full((r + 2, c), 5.0, dtype=torch.bfloat16, device="cuda") for r, c in shapes]
    b = zf.ortho_batch(xs, [o[1:-1] for o in outs])
    need = zf.orthogonalize_bytes(b)
    ws = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    zf.orthogonalize(b, ws[4096:4096 + need])
    torch.cuda.synchronize()
    assert (ws[:4096] == 0x5A).all() and (ws[4096 + need:] == 0x5A).all()
    for x, o in zip(xs, outs):
        assert (o[0] == 5.0).all() and (o[-1] == 5.0).all()
        assert off(o[1:-1], plain(x)) <= limit(1, torch.bfloat16)


def test_captured_and_replayed(zf):
    """Two graphs with workspaces of their own, replayed in turn with new
    inputs and eager work between: every replay equals the eager call."""
    shapes = [(256, 256), (100, 300), (17, 5)]
    sets = []
    for k in range(2):
        xs = [matrix(r, c, torch.float32, 20 + k) for r, c in shapes]
        ys = [torch.empty_like(x, dtype=torch.bfloat16) for x in xs]
        b = zf.ortho_batch(xs, ys)
        ws = torch.empty(zf.orthogonalize_bytes(b), dtype=torch.uint8, device="cuda")
        zf.orthogonalize(b, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            zf.orthogonalize(b, ws)
        sets.append((xs, ys, g, b, ws))
    for turn in range(4):
        for xs, ys, _, _, _ in sets:
            for i, x in enumerate(xs):
                x.copy_(matrix(*x.shape, torch.float32, 100 * turn + i))
            for y in ys:
                y.zero_()
        for _, _, g, _, _ in sets:
            g.replay()
        torch.cuda.synchronize()
        for xs, ys, _, _, _ in sets:
            eager = run(zf, xs, [torch.empty_like(y) for y in ys])
            for a, b in zip(ys, eager):
                assert torch.equal(G.bits_view(a), G.bits_view(b)), turn


def test_two_streams_at_once(zf):
    xs = [matrix(512, 768, torch.float32, k) for k in range(2)]
    want = [run(zf, [x], [torch.empty_like(x, dtype=torch.bfloat16)])[0] for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.empty_like(x, dtype=torch.bfloat16) for x in xs]
    bs = [zf.ortho_batch([x], [y]) for x, y in zip(xs, ys)]
    ws = [torch.empty(zf.orthogonalize_bytes(b), dtype=torch.uint8, device="cuda") for b in bs]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, w, st in zip(bs, ws, streams):
            zf.orthogonalize(b, w, stream=st)
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert torch.equal(G.bits_view(y), G.bits_view(w))


# ---- the Muon step ---------------------------------------------------------------

class Model:
    """Buffers of a step over segments (numel, unit, kind, rows), filled from
    a seed, with the same start for Muon and for the AdamW step."""

    def __init__(self, zf, segs, muon, n, layout, gdt="bf16", pdt="bf16", seed=1, scale=1.0,
                 dynamic=False, reduced=False):
        self.zf, self.segs, self.chosen, self.n = zf, segs, muon, n
        self.plan = zf.plan_flat(segs, n, layout, 2)
        self.muon = zf.muon_plan(self.plan, muon)
        self.gdt, self.pdt, self.scale = gdt, pdt, scale
        size = self.plan.psi_pad
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.real = torch.zeros(size, dtype=torch.bool, device="cuda")
        for u in self.plan.units:
            self.real[u.O:u.O + u.L] = True

        def normal(sigma):
            return torch.randn(size, generator=g, device="cuda") * sigma * self.real
        self.master, self.momentum = normal(0.02), normal(1e-3)
        self.square = normal(1e-3).square()
        self.grads = [(normal(1e-3) * scale).to(DT[gdt]) for _ in range(n)]
        self.params = self.master.to(DT[pdt]) if pdt else None
        self.shards = (torch.zeros(size, device="cuda")
                       if layout == W.PER_PARAM_DIM0 or reduced else None)
        self.reduced = reduced
        if reduced:
            total = self.grads[0].float()
            for q in self.grads[1:]:
                total = total + q.float()
            self.shards.copy_(total)
        self.state = torch.empty(zf.state_bytes(), dtype=torch.uint8, device="cuda")
        zf.state_init(self.state, scale, dynamic)
        self.workspace = torch.empty(zf.muon_workspace_bytes(self.muon), dtype=torch.uint8,
                                     device="cuda")
        self.workspace.fill_(0xFF)

    def places(self):
        """(first element, rows, cols) of the matrices."""
        lam, out = 0, []
        for i, (numel, _, _, rows) in enumerate(self.segs):
            if i in self.chosen:
                u = next(u for u in self.plan.units if u.lam <= lam < u.lam + u.L)
                out.append((u.O + lam - u.lam, rows, numel // rows))
            lam += numel
        return out

    def codes(self):
        code = {"f16": W.F16, "bf16": W.BF16, None: W.BF16}
        return code[self.gdt], code[self.pdt]

    def step(self, hp, mhp, stream=None):
        self.zf.muon_step(self.muon, hp, mhp, *self.codes(), None if self.reduced else self.grads,
                          self.master, self.momentum, self.square, self.params, self.workspace,
                          self.state, stream=stream, grad_shards=self.shards,
                          grads_reduced=self.reduced)

    def adamw(self, hp):
        self.zf.shard_step(self.plan, hp, *self.codes(), None if self.reduced else self.grads,
                           self.master, self.momentum, self.square, self.params, self.workspace,
                           self.state, grad_shards=self.shards, grads_reduced=self.reduced)

    def buffers(self):
        out = {"master": self.master, "momentum": self.momentum, "square": self.square,
               "state": self.state, "params": self.params, "shards": self.shards}
        return {k: v.clone() for k, v in out.items() if v is not None}


MLP = [(128 * 40, 0, 0, 128), (128, 0, 1, 0), (100 * 128, 1, 0, 100), (100, 1, 1, 0),
       (33 * 100, 2, 0, 33), (33, 2, 1, 0), (33 * 1, 3, 0, 33), (1, 3, 1, 0), (1 * 21, 4, 0, 1)]
MLP_MUON = [0, 2, 4, 6, 8]
WIDE = [(50 * 96, 0, 0, 50), (96 * 96, 1, 0, 96), (300 * 96, 1, 0, 300), (96 * 300, 1, 0, 96),
        (96, 1, 2, 0), (3, 1, 2, 0), (257 * 511, 2, 0, 257), (50 * 96, 2, 0, 50)]
WIDE_MUON = [6, 1, 2, 3]
# weights whose rows keep 16-byte alignment, of both orientations, and the same behind a vector of 3
EVEN = [(200 * 260, 0, 0, 200), (333 * 148, 0, 0, 333), (130 * 1028, 0, 0, 130),
        (3, 0, 2, 0), (200 * 260, 0, 0, 200), (333 * 148, 0, 0, 333)]
EVEN_MUON = [0, 1, 2, 4, 5]
THIN = [(1293 * 4, 0, 0, 1293), (1293, 0, 2, 0), (9 * 1293, 1, 0, 9), (300 * 700, 1, 0, 300)]

STEPS = [
    (EVEN, EVEN_MUON, 2, W.GLOBAL_FLAT, "bf16", "bf16", 1.0, True, "rms", False),
    (EVEN, EVEN_MUON, 4, W.PER_UNIT, "f16", "f16", 64.0, False, "rows", False),
    (EVEN, EVEN_MUON, 2, W.PER_PARAM_DIM0, "bf16", None, 1.0, True, "rms", False),
    (MLP, MLP_MUON, 4, W.PER_UNIT, "f16", "f16", 1024.0, True, "rms", False),
    (MLP, MLP_MUON, 1, W.GLOBAL_FLAT, "bf16", "bf16", 1.0, False, "rows", False),
    (MLP, MLP_MUON, 7, W.PER_PARAM_DIM0, "bf16", None, 1.0, True, "rows", False),
    (WIDE, WIDE_MUON, 2, W.GLOBAL_FLAT, "bf16", "f16", 1.0, True, "rms", False),
    (WIDE, WIDE_MUON, 9, W.PER_UNIT, "bf16", "bf16", 1.0, True, "rms", False),
    (WIDE, WIDE_MUON, 3, W.PER_PARAM_DIM0, "f16", "bf16", 256.0, False, "rms", True),
    (WIDE, WIDE_MUON, 5, W.PER_UNIT, "bf16", None, 1.0, True, "rows", True),
    (WIDE, list(range(4)), 2, W.GLOBAL_FLAT, "bf16", "bf16", 1.0, True, "rms", False),
]


@pytest.mark.parametrize("segs,muon,n,layout,gdt,pdt,scale,nesterov,rule,reduced", STEPS)
def test_muon_step(zf, segs, muon, n, layout, gdt, pdt, scale, nesterov, rule, reduced):
    """Three steps.  Sums, momentum and AdamW's part bit for bit; the
    matrices within the iteration's tolerance of the update's size."""
    kw = dict(gdt=gdt, pdt=pdt, scale=scale, reduced=reduced)
    a, twin = (Model(zf, segs, muon, n, layout, **kw) for _ in range(2))
    lr, mlr, mu, decay = 2e-3, 1e-2, 0.9, 0.1
    hp = zf.hparams(lr, weight_decay=0.01, max_norm=0.05)
    mhp = zf.muon_hparams(mlr, momentum=mu, weight_decay=decay, nesterov=nesterov,
                          scale_rule=zf.MUON_SCALE_RMS if rule == "rms" else zf.MUON_SCALE_ROWS)
    matrices = torch.zeros_like(a.real)
    for at, r, c in a.places():
        matrices[at:at + r * c] = True
    for k in range(3):
        before = a.buffers()
        for name in ("master", "momentum", "square"):  # AdamW from the same state
            getattr(twin, name).copy_(before[name])
        a.step(hp, mhp)
        twin.adamw(hp)
        res, ref = zf.read_result(a.state), zf.read_result(twin.state)
        assert (res.t, res.gs, res.skipped) == (ref.t, ref.gs, ref.skipped) == (k + 1, ref.gs, 0)
        after, other = a.buffers(), twin.buffers()
        for name in ("master", "momentum", "square", "params"):
            if name in after:
                assert torch.equal(G.bits_view(after[name][~matrices]),
                                   G.bits_view(other[name][~matrices])), name
        assert torch.equal(after["square"][matrices], before["square"][matrices])
        if a.shards is not None:
            assert torch.equal(after["shards"], other["shards"])
        total = a.shards
        if total is None:
            total = a.grads[0].float()
            for q in a.grads[1:]:
                total = total + q.float()
        g = total * torch.tensor(res.gs, device="cuda")
        moment = torch.tensor(mu, device="cuda") * before["momentum"] + g
        assert torch.equal(after["momentum"][matrices], moment[matrices])
        u = g + torch.tensor(mu, device="cuda") * moment if nesterov else moment
        for at, r, c in a.places():
            p = slice(at, at + r * c)
            o = plain(u[p].view(r, c)).reshape(-1)
            rate = mlr * (0.2 * math.sqrt(max(r, c)) if rule == "rms"
                          else math.sqrt(max(1.0, r / c)))
            want = before["master"][p].double() * (1 - mlr * decay) - rate * o
            # four roundings of 2^-24 (the factor, two products, the difference)
            room = TOL[1] * rate * o.norm() + 4 * 2.0 ** -24 * (want.norm() + rate * o.norm())
            assert (after["master"][p].double() - want).norm() <= room, (k, r, c)
            if a.params is not None:
                assert torch.equal(after["params"][p], after["master"][p].to(a.params.dtype))


def test_few_thin_blocks_take_three_products(zf):
    """Less than a round of blocks, thin ones too long for shared memory among
    them."""
    m = Model(zf, THIN, [0, 2, 3], 2, W.GLOBAL_FLAT)
    before = m.buffers()
    mhp = zf.muon_hparams(0.5, momentum=0.9, weight_decay=0.0, nesterov=False,
                          scale_rule=zf.MUON_SCALE_ROWS)
    m.step(zf.hparams(1e-3, max_norm=0.0), mhp)
    for at, r, c in m.places():
        p = slice(at, at + r * c)
        o = plain(m.momentum[p].view(r, c)).reshape(-1)
        rate = 0.5 * math.sqrt(max(1.0, r / c))
        want = before["master"][p].double() - rate * o
        room = TOL[3] * rate * o.norm() + 4 * 2.0 ** -24 * (want.norm() + rate * o.norm())
        assert (m.master[p].double() - want).norm() <= room, (r, c)


def test_padding_stays_zero(zf):
    m = Model(zf, MLP, MLP_MUON, 7, W.PER_PARAM_DIM0)
    m.step(zf.hparams(1e-3), zf.muon_hparams(1e-2))
    for t in (m.master, m.momentum, m.square, m.params, m.shards):
        assert (t[~m.real] == 0).all()


@pytest.mark.parametrize("value", ["inf", "nan"])
@pytest.mark.parametrize("where", [0, 128 * 40 + 5])
def test_overflow_skips_everything(zf, value, where):
    m = Model(zf, MLP, MLP_MUON, 3, W.GLOBAL_FLAT, gdt="f16", pdt="f16", scale=1024.0,
              dynamic=True)
    m.grads[1][where] = float(value)
    before = m.buffers()
    m.step(zf.hparams(1e-3), zf.muon_hparams(1e-2))
    res = zf.read_result(m.state)
    assert (res.skipped, res.t, res.scale_next) == (1, 0, 512.0)
    after = m.buffers()
    for name in ("master", "momentum", "square", "params"):
        assert torch.equal(G.bits_view(after[name]), G.bits_view(before[name])), name


def test_three_products_in_the_step(zf):
    m = Model(zf, WIDE, WIDE_MUON, 2, W.GLOBAL_FLAT)
    ns = zf.ns_params(products=3)
    m.workspace = torch.empty(zf.muon_workspace_bytes(m.muon, ns), dtype=torch.uint8,
                              device="cuda")
    before = m.buffers()
    mhp = zf.muon_hparams(0.5, momentum=0.9, weight_decay=0.0, nesterov=False,
                          scale_rule=zf.MUON_SCALE_ROWS, ns=ns)
    m.step(zf.hparams(1e-3, max_norm=0.0), mhp)
    for at, r, c in m.places():
        p = slice(at, at + r * c)
        o = plain(m.momentum[p].view(r, c)).reshape(-1)
        rate = 0.5 * math.sqrt(max(1.0, r / c))
        want = before["master"][p].double() - rate * o
        room = TOL[3] * rate * o.norm() + 4 * 2.0 ** -24 * (want.norm() + rate * o.norm())
        assert (m.master[p].double() - want).norm() <= room


def test_step_captured_and_replayed(zf):
    """A graph of the step replayed beside an eager twin, with new gradients
    between replays and one overflow among them."""
    kw = dict(gdt="f16", pdt="f16", scale=1024.0, dynamic=True)
    a, b = (Model(zf, WIDE, WIDE_MUON, 2, W.PER_UNIT, **kw) for _ in range(2))
    hp, mhp = zf.hparams(1e-3), zf.muon_hparams(1e-2)
    for m in (a, b):
        m.step(hp, mhp)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(hp, mhp)
    g = torch.Generator(device="cuda").manual_seed(77)
    for k in range(5):
        for q, r in zip(a.grads, b.grads):
            new = (torch.randn(q.shape, generator=g, device="cuda") * a.real).to(q.dtype)
            if k == 2:
                new[10] = float("inf")
            q.copy_(new)
            r.copy_(new)
        graph.replay()
        b.step(hp, mhp)
        torch.cuda.synchronize()
        x, y = a.buffers(), b.buffers()
        for name in x:
            assert torch.equal(x[name].view(torch.uint8), y[name].view(torch.uint8)), (k, name)
    assert zf.read_result(a.state).t == 5


def test_step_workspace_guards(zf):
    m = Model(zf, WIDE, WIDE_MUON, 9, W.PER_UNIT)
    need = zf.muon_workspace_bytes(m.muon)
    ws = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    m.workspace = ws[4096:4096 + need]
    m.step(zf.hparams(1e-3), zf.muon_hparams(1e-2))
    torch.cuda.synchronize()
    assert (ws[:4096] == 0x5A).all() and (ws[4096 + need:] == 0x5A).all()


def test_accumulated_buckets_then_muon(zf):
    """The calls as a training loop makes them: micro-batches reduce-scattered
    into the shards, a Muon step on them, the orthogonalised momentum of one
    matrix alone, and the unit gather of the new parameters."""
    m = Model(zf, WIDE, WIDE_MUON, 2, W.PER_UNIT, reduced=True)
    for micro in range(2):
        for g in range(len(m.plan.groups)):
            zf.bucket_reduce_scatter(m.plan, g, W.BF16, m.grads, m.shards, micro > 0)
    before = m.buffers()
    mhp = zf.muon_hparams(1e-2, nesterov=False, weight_decay=0.0)
    m.step(zf.hparams(1e-3), mhp)
    at, r, c = m.places()[0]
    p = slice(at, at + r * c)
    alone = torch.empty(r, c, device="cuda")
    # a matrix held in shared memory takes three products in a step
    run(zf, [m.momentum[p].view(r, c)], [alone], zf.ns_params(products=3))
    rate = torch.tensor(1e-2 * 0.2 * math.sqrt(max(r, c)), dtype=torch.float64).float().cuda()
    want = before["master"][p] - rate * alone.reshape(-1)
    assert torch.equal(m.master[p], want)
    u = m.plan.units[1]
    shards = [m.params[u.O + k * u.S:u.O + (k + 1) * u.S] for k in range(2)]
    buf = torch.empty(u.P, dtype=m.params.dtype, device="cuda")
    zf.gather(m.plan, 1, W.BF16, shards, buf)
    assert torch.equal(G.bits_view(buf), G.bits_view(m.params[u.O:u.O + u.P]))
