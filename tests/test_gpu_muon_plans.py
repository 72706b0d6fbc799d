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
