"""Limits of a rank's forward and backward calls, as the header states them (no GPU needed: every call returns before
the HIP runtime is touched)."""
import ctypes as C
import os
import re

import pytest

from tests import test_rank_ops_cpu as calls

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def zf():
    from fsdp_sharded_mixed_amd import zf as Z
    return Z


def stated(name):
    """A limit of the header, `1ll << n`."""
    with open(os.path.join(ROOT, "include", "zf.h")) as f:
        return 1 << int(re.search(rf"#define {name} \(\(1ll << (\d+)\)\)", f.read()).group(1))


@pytest.mark.parametrize("call,key", [
    ("embedding", "out_stride"), ("embedding_grad", "dout_stride"), ("layer_norm", "x_stride"),
    ("layer_norm", "y_stride"), ("layer_norm_grad", "dy_stride"), ("layer_norm_grad", "x_stride"),
    ("layer_norm_grad", "dx_stride"), ("weight_grad", "dy_stride")])
def test_strides(zf, call, key):
    assert getattr(calls, call)(zf, **{key: stated("ZF_MAX_STRIDE") + 1}) == "ZF_ESIZE"


@pytest.mark.parametrize("key", ["code_stride", "scale_stride"])
def test_strides_of_checkpoints(zf, key):
    a = calls.act8(zf, **{key: stated("ZF_MAX_STRIDE") + 1})
    for fn in (zf.lib.zf_act8_store, zf.lib.zf_act8_load):
        assert zf.STATUS[fn(C.byref(a), zf.BF16, calls.BASE, 64, None)] == "ZF_ESIZE"
    assert calls.layer_norm(zf, x8=a) == calls.layer_norm(zf, y8=a) == "ZF_ESIZE"
    assert calls.layer_norm_grad(zf, x=None, x8=a) == calls.weight_grad(zf, x8=a) == "ZF_ESIZE"


@pytest.mark.parametrize("name,sizes", [
    ("embedding_grad_bytes", [(40960, 1024), (32000, 2048), (1, 8), (300001, 24), (511, 65), (1000, 8192), (97, 1 << 20)]),
    ("layer_norm_grad_bytes", [(1024,), (40,), (2049,), (10000,), (16385,)]),
    ("weight_grad_bytes", [(256, 1024), (1024, 1024), (2048, 2048), (777, 1000), (1, 1), (8192, 2048), (2049, 2047),
                           (4, 1 << 20)])])
def test_a_longer_batch_has_a_workspace_for_every_shorter_one(zf, name, sizes):
    """A program keeps one workspace for its longest batch: sizes never fall as batches grow."""
    fn = getattr(zf.lib, "zf_" + name)
    for size in sizes:
        most = 0
        batches = list(range(0, 40000, 7)) + [k << e for e in range(15, 29) for k in (1, 3)]
        batches = sorted(set(batches + [b + d for b in batches[-30:] for d in (-1, 1)]))
        for rows in batches:
            need = fn(rows, *size)
            assert need >= most, f"{size}: {rows} rows need {need} bytes, fewer {most}"
            most = need
