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
