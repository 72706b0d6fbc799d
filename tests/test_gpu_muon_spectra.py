"""Orthogonalisation of matrices whose singular values differ by orders of
magnitude, against the plain form in 64 bits.

Tolerances, in |error|_F / |X|_F, f the map of all steps on singular values.

One product.  u = 2^-11 is half a step of an operand.  To first order an error
W (in the singular vectors' basis) that arises in X reaches the result as
W_ij times a divided difference of f: at most (f_i + f_j) / (s_i + s_j) where
s_i and s_j differ, a^steps for two small ones.  An error of B = b A + c A A,
E, arises as W_ij = E_ij s_j, one of X's rounding in B X as W_ij = B_i d_ij
with B_i <= 4.8 s_i^2: both have a factor that cancels the division, so that
neither grows while the small singular values do.  Every other term must keep
more bits than that growth (a^5 = 485 for the default steps) costs: X itself
has 22.  What then arises is the sum over the steps of at most (3.5 + 2 +
4.8 * 3 * 1.2) u = 23 u if all roundings are aligned; they are spread evenly
(0.41 u in the mean over a binade), and the last factor is near 0.7 where the
singular values end: 3.4 u a step, of which two steps' worth survives near 1.
7 u = 3.4e-3, taken as 2^-8.

Three products.  X is kept to 22 bits (an error of 0.41 * 2^-22 of its norm 1
in the mean), and every addition of a sum rounds to 24 (0.41 * 2^-24 of the
partial sum, which grows evenly to the whole one: sqrt(k / 3) for k terms).
Both arise anywhere, so both grow with the smallest singular values, a^5 over
a result whose norm is 0.68 at least, and arise anew in every step, 1 + 1/a +
1/a^2 + ... = 1.41 in all.  An error of the long sums in A does not grow; those
of B X have min(rows, cols) terms.  (The same iteration in 32-bit arithmetic
has errors of this size.)
"""
import math

import pytest
import torch

from tests import gpu_common as G
from tests.test_gpu_muon import plain, off, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    from fsdp_sharded_mixed_amd import zf as Z
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return Z


def tolerance(products, rows, cols, steps=5):
    if products == 1:
        return 2.0 ** -8
    noise = 0.41 * (2.0 ** -22 + 2.0 ** -24 * math.sqrt(min(rows, cols) / 3))
    return max(2e-5, 1.41 / 0.68 * 3.4445 ** steps * noise)


def spectrum(kind, rows, cols, seed):
    """One strong direction over noise, half the directions over noise, or nine
    in ten of equal strength."""
    g = torch.Generator().manual_seed(seed)
    noise = torch.randn(rows, cols, generator=g)
    if kind == "half":
        r = max(1, min(rows, cols) // 2)
        strong = torch.randn(rows, r, generator=g) @ torch.randn(r, cols, generator=g) / math.sqrt(r)
        return strong + 1e-3 * noise
    if kind == "equal":
        r = max(1, min(rows, cols) * 9 // 10)
        left = torch.linalg.qr(torch.randn(rows, r, generator=g))[0]
        right = torch.linalg.qr(torch.randn(cols, r, generator=g))[0]
        return left @ right.t() + 1e-4 * noise / math.sqrt(max(rows, cols))
    strong = torch.randn(rows, 1, generator=g) @ torch.randn(1, cols, generator=g)
    return strong + float(kind) * noise


KINDS = ["0", "1e-4", "1e-3", "1e-2", "half", "equal"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(11, 2000), (1400, 64), (256, 1024), (600, 600), (4, 1293),
                                       (32, 600), (100, 128)])
@pytest.mark.parametrize("products", [1, 3])
def test_strong_directions(zf, kind, rows, cols, products):
    """Alone, and in a batch of more than 256 blocks of 64 x 64 (or 24)."""
    blocks = -(-rows // 64) * -(-cols // 64)
    xs = [spectrum(kind, rows, cols, k).cuda() for k in range(min(256 // blocks + 1, 24))]
    want = [plain(x) for x in xs]
    for n in (1, len(xs)):
        ys = run(zf, xs[:n], [torch.empty_like(x) for x in xs[:n]], zf.ns_params(products=products))
        worst = max(off(y, w) for y, w in zip(ys, want))
        G.say(f"{kind} {rows}x{cols} products={products} of {n}: {worst:.2e}")
        assert worst <= tolerance(products, rows, cols)


@pytest.mark.parametrize("rows,cols", [(1024, 1024), (2000, 2048), (2048, 1024),
                                       (1024, 4096)])
@pytest.mark.parametrize("kind", ["0", "1e-3", "half"])
def test_strong_directions_of_a_layer(zf, kind, rows, cols):
    """Larger matrices in the default mode, from and to bf16."""
    xs = [spectrum(kind, rows, cols, k).cuda().bfloat16() for k in range(2)]
    ys = run(zf, xs, [torch.empty_like(x) for x in xs])
    worst = max(off(y, plain(x)) for x, y in zip(xs, ys))
    G.say(f"{kind} {rows}x{cols}: {worst:.2e}")
    assert worst <= tolerance(1, rows, cols) + torch.finfo(torch.bfloat16).eps / 2


@pytest.mark.parametrize("dst", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(300, 2500), (1293, 4), (1024, 1024), (90, 70)])
@pytest.mark.parametrize("large", [9, 36])
def test_alone_and_among_others(zf, shape, large, dst):
    """The same bits whatever else is in the call (36: blocks of the first
    launches take 4 tiles each)."""
    x = spectrum("half", *shape, 3).cuda()
    others = [spectrum("1e-2", *s, k % 5).cuda()
              for k, s in enumerate([(256, 2048)] * large + [(20, 30)] * 15)]
    alone = run(zf, [x], [torch.empty_like(x, dtype=dst)])[0]
    xs = others + [x]
    among = run(zf, xs, [torch.empty_like(z, dtype=dst) for z in xs])[-1]
    assert torch.equal(G.bits_view(alone), G.bits_view(among))


@pytest.mark.parametrize("shape", [(1, 77), (65, 1), (1, 1000), (3000, 1), (1, 8191)])
def test_rows_and_columns_with_one_product(zf, shape):
    """One singular value s, A = |hi|^2 the only inexact number: off by 2 * 0.41
    * 2^-11 / sqrt(n / 3) in the mean for n normal elements, so under 1e-4 a
    step, of which five steps at a slope of up to 1.7 make 7e-4: 2^-10."""
    for seed in range(5):
        x = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()
        y = run(zf, [x], [torch.empty_like(x)], zf.ns_params(products=1))[0]
        err = off(y, plain(x))
        G.say(f"{shape}: {err:.2e}")
        assert err <= 2.0 ** -10


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes_and_kinds(zf, seed):
    """Sparse matrices, rows of different scales, one large element and random
    ranks over noise, in batches of random shapes."""
    g = torch.Generator().manual_seed(1000 + seed)

    def number(lo, hi):
        return int(round(math.exp(math.log(lo) + math.log(hi / lo) * torch.rand(1, generator=g).item())))
    xs = []
    for k in range(12):
        r, c = number(1, 1500), number(1, 2500)
        x = torch.randn(r, c, generator=g)
        if k % 4 == 0:
            x = x * (torch.rand(r, c, generator=g) < 0.02)
            x[number(1, r) - 1, 0] = 1.0
        elif k % 4 == 1:
            x = x * 10 ** (-3 * torch.rand(r, 1, generator=g))
        elif k % 4 == 2:
            x[0, 0] *= 1000.0
        else:
            n = number(1, min(r, c))
            x = torch.randn(r, n, generator=g) @ torch.randn(n, c, generator=g) + 1e-3 * x
        xs.append(x.cuda())
    for products in (1, 3):
        ys = run(zf, xs, [torch.empty_like(x) for x in xs], zf.ns_params(products=products))
        for x, y in zip(xs, ys):
            err = off(y, plain(x))
            G.say(f"{tuple(x.shape)} products={products}: {err:.2e}")
            assert err <= tolerance(products, *x.shape), tuple(x.shape)
