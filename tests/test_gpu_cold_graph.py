"""A rank's forward and backward calls captured in a process that has run none of their kernels before."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

CHILD = """
import torch
from fsdp_sharded_mixed_amd import zf
t, v, h, o = 5000, 300, 512, 256
g = torch.Generator(device="cuda").manual_seed(1)
def normal(*shape):
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)
def zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")
def blank():
    return zf.act8(zeros(t, h, dtype=torch.uint8), zeros(t, h // 32, dtype=torch.uint8))
table, w, dy, dout = normal(v, h), normal(h), normal(t, h), normal(t, o)
ids = torch.randint(-1, v, (t,), device="cuda", generator=g)
x, y, dx, back = (zeros(t, h, dtype=torch.bfloat16) for _ in range(4))
mean, rstd, dw, db, dt, dl = zeros(t), zeros(t), zeros(h), zeros(h), zeros(v, h), zeros(o, h)
x8, y8, dx8 = blank(), blank(), blank()
ws = zeros(max(zf.embedding_grad_bytes(t, v, h), zf.layer_norm_grad_bytes(t, h), zf.weight_grad_bytes(t, o, h)),
           dtype=torch.uint8)
outs = [x, y, dx, back, mean, rstd, dw, db, dt, dl, x8.codes, y8.codes, dx8.codes]
def run():
    zf.embedding(table, ids, x)
    zf.layer_norm(zf.NORM_LAYER, x, w, w, 1e-5, y, mean, rstd, x8=x8, y8=y8)
    zf.weight_grad(dout, y8, dl, ws)
    zf.layer_norm_grad(zf.NORM_LAYER, dy, x8, w, mean, rstd, dx, dw, db, ws)
    zf.embedding_grad(dx, ids, dt, ws)
    zf.act8_store(dx8, dx)
    zf.act8_load(dx8, back)
def taken():
    torch.cuda.synchronize()
    got = [z.clone() for z in outs]
    for z in outs:
        z.zero_()
    return got
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
got = [taken()]
graph.replay()
got.append(taken())
run()
want = taken()
assert all(bool((z != 0).any()) for z in want)
assert all(torch.equal(a, b) for k in got for a, b in zip(k, want))
print("the same")
"""


def test_captured_before_any_other_run():
    done = subprocess.run([sys.executable, "-c", CHILD], cwd=Path(__file__).parent.parent, capture_output=True, text=True,
                          timeout=100)
    assert done.returncode == 0 and "the same" in done.stdout, done.stderr[-2000:]
