"""Argument checks of a rank's forward and backward calls (no GPU needed): every call here returns before the HIP
runtime is touched, and leaves nothing enqueued.  Device addresses are made-up numbers that no kernel sees."""
import ctypes as C

import pytest
import torch

from tests import rank_ops as R

BASE = 1 << 20
BIG = 1 << 50


@pytest.fixture(scope="module")
def zf():
    from fsdp_sharded_mixed_amd import zf as Z
    return Z


def act8(zf, rows=8, cols=64, **kw):
    f = dict(codes=11 * BASE, scales=12 * BASE, rows=rows, cols=cols, code_stride=cols, scale_stride=-(-cols // 32))
    f.update(kw)
    return zf.Act8Struct(**f)


def embedding(zf, **kw):
    f = dict(table_dtype=zf.BF16, dtype=zf.BF16, id_bytes=4, scale=1.0, tokens=8, vocab=100, cols=64, ids=BASE,
             table=2 * BASE, out=3 * BASE, out_stride=64)
    f.update(kw)
    return zf.STATUS[zf.lib.zf_embedding(C.byref(zf.EmbeddingArgs(**f)), None)]


def embedding_grad(zf, **kw):
    f = dict(dtype=zf.BF16, grad_dtype=zf.F32, id_bytes=4, accumulate=0, scale=1.0, reserved=0, tokens=8, vocab=100,
             cols=64, ids=BASE, dout=2 * BASE, dout_stride=64, grad=3 * BASE, workspace=4 * BASE, workspace_size=BIG)
    f.update(kw)
    return zf.STATUS[zf.lib.zf_embedding_grad(C.byref(zf.EmbeddingGradArgs(**f)), None)]


def layer_norm(zf, **kw):
    f = dict(kind=zf.NORM_LAYER, dtype=zf.BF16, weight_dtype=zf.BF16, reserved=0, eps=1e-5, rows=8, cols=64, x=BASE,
             x_stride=64, weight=2 * BASE, bias=3 * BASE, y=4 * BASE, y_stride=64, mean=5 * BASE, rstd=6 * BASE)
    f.update(kw)
    for key in ("x8", "y8"):
        f[key] = C.pointer(f[key]) if f.get(key) else None
    return zf.STATUS[zf.lib.zf_layer_norm(C.byref(zf.LayerNormArgs(**f)), None)]


def layer_norm_grad(zf, **kw):
    f = dict(kind=zf.NORM_LAYER, dtype=zf.BF16, weight_dtype=zf.BF16, grad_dtype=zf.F32, accumulate=0, reserved=0,
             rows=8, cols=64, dy=BASE, dy_stride=64, x=2 * BASE, x_stride=64, weight=3 * BASE, mean=4 * BASE,
             rstd=5 * BASE, dx=6 * BASE, dx_stride=64, weight_grad=7 * BASE, bias_grad=8 * BASE, workspace=9 * BASE,
             workspace_size=BIG)
    f.update(kw)
    f["x8"] = C.pointer(f["x8"]) if f.get("x8") else None
    return zf.STATUS[zf.lib.zf_layer_norm_grad(C.byref(zf.LayerNormGradArgs(**f)), None)]


def weight_grad(zf, **kw):
    f = dict(dtype=zf.BF16, grad_dtype=zf.F32, accumulate=0, reserved=0, rows=8, out_features=16, in_features=64,
             dy=BASE, dy_stride=16, grad=2 * BASE, workspace=3 * BASE, workspace_size=BIG)
    x8 = act8(zf)
    f.update(x8=x8)
    f.update(kw)
    f["x8"] = C.pointer(f["x8"]) if f["x8"] else None
    return zf.STATUS[zf.lib.zf_weight_grad(C.byref(zf.WeightGradArgs(**f)), None)]


ROWS_MAX, COLS_MAX = 1 << 30, 1 << 20


@pytest.mark.parametrize("kw,want", [
    ({"ids": None}, "ZF_EINVAL"), ({"table": None}, "ZF_EINVAL"), ({"out": None}, "ZF_EINVAL"),
    ({"id_bytes": 2}, "ZF_EINVAL"), ({"tokens": -1}, "ZF_EINVAL"), ({"vocab": 0}, "ZF_EINVAL"),
    ({"cols": 0}, "ZF_EINVAL"), ({"out_stride": 63}, "ZF_EINVAL"), ({"dtype": 4}, "ZF_EDTYPE"),
    ({"table_dtype": 0}, "ZF_EDTYPE"), ({"ids": BASE + 2}, "ZF_EALIGN"),
    ({"id_bytes": 8, "ids": BASE + 4}, "ZF_EALIGN"), ({"table": BASE + 1}, "ZF_EALIGN"),
    ({"out": BASE + 1}, "ZF_EALIGN"), ({"tokens": ROWS_MAX + 1}, "ZF_ESIZE"), ({"vocab": ROWS_MAX + 1}, "ZF_ESIZE"),
    ({"cols": COLS_MAX + 1}, "ZF_ESIZE"), ({"out_stride": 1 << 40}, "ZF_ESIZE"),
    ({"tokens": 0, "ids": None, "out": None, "table": None}, "ZF_OK")])
def test_embedding(zf, kw, want):
    assert embedding(zf, **kw) == want


@pytest.mark.parametrize("kw,want", [
    ({"ids": None}, "ZF_EINVAL"), ({"dout": None}, "ZF_EINVAL"), ({"grad": None}, "ZF_EINVAL"),
    ({"workspace": None}, "ZF_EINVAL"), ({"accumulate": 2}, "ZF_EINVAL"), ({"reserved": 1}, "ZF_EINVAL"),
    ({"id_bytes": 0}, "ZF_EINVAL"), ({"tokens": -1}, "ZF_EINVAL"), ({"vocab": 0}, "ZF_EINVAL"),
    ({"cols": -3}, "ZF_EINVAL"), ({"dout_stride": 1}, "ZF_EINVAL"), ({"dtype": 9}, "ZF_EDTYPE"),
    ({"grad_dtype": 9}, "ZF_EDTYPE"), ({"dout": BASE + 1}, "ZF_EALIGN"), ({"grad": BASE + 2}, "ZF_EALIGN"),
    ({"workspace": BASE + 8}, "ZF_EALIGN"), ({"workspace_size": 100}, "ZF_ESIZE"),
    ({"tokens": ROWS_MAX + 1}, "ZF_ESIZE"), ({"cols": COLS_MAX + 1}, "ZF_ESIZE"),
    ({"tokens": 0, "ids": None, "dout": None, "workspace": None, "workspace_size": 0, "accumulate": 1}, "ZF_OK")])
def test_embedding_grad(zf, kw, want):
    assert embedding_grad(zf, **kw) == want


def test_embedding_grad_bytes(zf):
    assert zf.embedding_grad_bytes(0, 100, 64) == 0
    sizes = [zf.embedding_grad_bytes(n, 40960, 2048) for n in (1, 100, 5000, 32768, 1 << 22)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    for args in ((-1, 100, 64), (8, 0, 64), (8, 100, 0)):
        with pytest.raises(zf.ZfError) as e:
            zf.embedding_grad_bytes(*args)
        assert zf.STATUS[e.value.status] == "ZF_EINVAL"


@pytest.mark.parametrize("kw,want", [
    ({"rows": -1}, "ZF_EINVAL"), ({"cols": 0}, "ZF_EINVAL"), ({"codes": None}, "ZF_EINVAL"),
    ({"scales": None}, "ZF_EINVAL"), ({"code_stride": 63}, "ZF_EINVAL"), ({"scale_stride": 1}, "ZF_EINVAL"),
    ({"rows": ROWS_MAX + 1}, "ZF_ESIZE"), ({"cols": COLS_MAX + 1, "code_stride": BIG}, "ZF_ESIZE"),
    ({"code_stride": 1 << 40}, "ZF_ESIZE"), ({"rows": 0, "codes": None, "scales": None}, "ZF_OK")])
def test_checkpoint_buffers(zf, kw, want):
    for fn in (zf.lib.zf_act8_store, zf.lib.zf_act8_load):
        assert zf.STATUS[fn(C.byref(act8(zf, **kw)), zf.BF16, BASE, 64, None)] == want


@pytest.mark.parametrize("dtype,x,stride,want", [
    (0, BASE, 64, "ZF_EDTYPE"), (2, None, 64, "ZF_EINVAL"), (2, BASE + 1, 64, "ZF_EALIGN"),
    (3, BASE + 2, 64, "ZF_EALIGN"), (2, BASE, 63, "ZF_EINVAL")])
def test_checkpoint_rows(zf, dtype, x, stride, want):
    for fn in (zf.lib.zf_act8_store, zf.lib.zf_act8_load):
        assert zf.STATUS[fn(C.byref(act8(zf)), dtype, x, stride, None)] == want
    assert zf.STATUS[zf.lib.zf_act8_store(None, 2, BASE, 64, None)] == "ZF_EINVAL"


@pytest.mark.parametrize("kw,want", [
    ({"kind": 2}, "ZF_EINVAL"), ({"reserved": 1}, "ZF_EINVAL"), ({"eps": -1e-9}, "ZF_EINVAL"),
    ({"eps": float("nan")}, "ZF_EINVAL"), ({"eps": float("inf")}, "ZF_EINVAL"), ({"x": None}, "ZF_EINVAL"),
    ({"y": None}, "ZF_EINVAL"), ({"weight": None}, "ZF_EINVAL"), ({"mean": None}, "ZF_EINVAL"),
    ({"rstd": None}, "ZF_EINVAL"), ({"rows": -1}, "ZF_EINVAL"), ({"cols": 0}, "ZF_EINVAL"),
    ({"x_stride": 63}, "ZF_EINVAL"), ({"y_stride": 63}, "ZF_EINVAL"),
    ({"y": BASE, "y_stride": 65}, "ZF_EINVAL"), ({"dtype": 7}, "ZF_EDTYPE"), ({"weight_dtype": 0}, "ZF_EDTYPE"),
    ({"x": BASE + 1}, "ZF_EALIGN"), ({"y": BASE + 1}, "ZF_EALIGN"), ({"weight": BASE + 1}, "ZF_EALIGN"),
    ({"bias": BASE + 1}, "ZF_EALIGN"), ({"mean": BASE + 2}, "ZF_EALIGN"), ({"rstd": BASE + 2}, "ZF_EALIGN"),
    ({"rows": ROWS_MAX + 1}, "ZF_ESIZE"), ({"cols": COLS_MAX + 1}, "ZF_ESIZE"),
    ({"rows": 0, "x": None, "y": None, "weight": None, "mean": None, "rstd": None}, "ZF_OK")])
def test_layer_norm(zf, kw, want):
    assert layer_norm(zf, **kw) == want


def test_layer_norm_checkpoints(zf):
    for key in ("x8", "y8"):
        assert layer_norm(zf, **{key: act8(zf, cols=63)}) == "ZF_EINVAL"
        assert layer_norm(zf, **{key: act8(zf, rows=7)}) == "ZF_EINVAL"
        assert layer_norm(zf, **{key: act8(zf, codes=None)}) == "ZF_EINVAL"


@pytest.mark.parametrize("kw,want", [
    ({"kind": -1}, "ZF_EINVAL"), ({"reserved": 1}, "ZF_EINVAL"), ({"accumulate": -1}, "ZF_EINVAL"),
    ({"dy": None}, "ZF_EINVAL"), ({"x": None}, "ZF_EINVAL"), ({"dx": None}, "ZF_EINVAL"),
    ({"weight": None}, "ZF_EINVAL"), ({"mean": None}, "ZF_EINVAL"), ({"rstd": None}, "ZF_EINVAL"),
    ({"workspace": None}, "ZF_EINVAL"), ({"rows": -2}, "ZF_EINVAL"), ({"cols": 0}, "ZF_EINVAL"),
    ({"dy_stride": 63}, "ZF_EINVAL"), ({"x_stride": 63}, "ZF_EINVAL"), ({"dx_stride": 63}, "ZF_EINVAL"),
    ({"dx": BASE, "dx_stride": 70}, "ZF_EINVAL"), ({"dtype": 5}, "ZF_EDTYPE"), ({"weight_dtype": 5}, "ZF_EDTYPE"),
    ({"grad_dtype": 5}, "ZF_EDTYPE"), ({"dy": BASE + 1}, "ZF_EALIGN"), ({"x": BASE + 1}, "ZF_EALIGN"),
    ({"dx": BASE + 1}, "ZF_EALIGN"), ({"weight_grad": BASE + 2}, "ZF_EALIGN"),
    ({"bias_grad": BASE + 2}, "ZF_EALIGN"), ({"workspace": BASE + 4}, "ZF_EALIGN"),
    ({"workspace_size": 0}, "ZF_ESIZE"), ({"rows": ROWS_MAX + 1}, "ZF_ESIZE"),
    ({"cols": COLS_MAX + 1}, "ZF_ESIZE")])
def test_layer_norm_grad(zf, kw, want):
    assert layer_norm_grad(zf, **kw) == want


def test_layer_norm_grad_takes_x_or_its_checkpoint(zf):
    assert layer_norm_grad(zf, x8=act8(zf)) == "ZF_EINVAL"  # both
    assert layer_norm_grad(zf, x=None, x8=act8(zf, rows=9)) == "ZF_EINVAL"
    assert layer_norm_grad(zf, x=None, x8=act8(zf, scales=None)) == "ZF_EINVAL"
    nothing = dict(rows=0, dy=None, x=None, dx=None, weight=None, mean=None, rstd=None)
    assert layer_norm_grad(zf, **nothing, weight_grad=None, bias_grad=None) == "ZF_OK"


@pytest.mark.parametrize("kw,want", [
    ({"dy": None}, "ZF_EINVAL"), ({"x8": None}, "ZF_EINVAL"), ({"grad": None}, "ZF_EINVAL"),
    ({"accumulate": 3}, "ZF_EINVAL"), ({"reserved": 2}, "ZF_EINVAL"), ({"rows": -1}, "ZF_EINVAL"),
    ({"rows": 9}, "ZF_EINVAL"), ({"in_features": 65}, "ZF_EINVAL"), ({"out_features": 0}, "ZF_EINVAL"),
    ({"dy_stride": 15}, "ZF_EINVAL"), ({"dtype": 3}, "ZF_EDTYPE"), ({"grad_dtype": 0}, "ZF_EDTYPE"),
    ({"dy": BASE + 1}, "ZF_EALIGN"), ({"grad": BASE + 2}, "ZF_EALIGN"), ({"workspace": BASE + 8}, "ZF_EALIGN"),
    ({"out_features": COLS_MAX + 1, "dy_stride": BIG}, "ZF_ESIZE"), ({"dy_stride": 1 << 40}, "ZF_ESIZE")])
def test_weight_grad(zf, kw, want):
    assert weight_grad(zf, **kw) == want


def test_weight_grad_workspace(zf):
    need = zf.weight_grad_bytes(1 << 14, 256, 1024)
    assert need > 0
    long = dict(rows=1 << 14, out_features=256, in_features=1024, dy_stride=256)
    x8 = act8(zf, 1 << 14, 1024)
    assert weight_grad(zf, **long, x8=x8, workspace_size=need - 1) == "ZF_ESIZE"
    assert weight_grad(zf, **long, x8=x8, workspace=None) == "ZF_EINVAL"
    nothing = dict(rows=0, x8=act8(zf, 0), dy=None, workspace=None, workspace_size=0)
    assert weight_grad(zf, **nothing, accumulate=1) == "ZF_OK"


def test_the_binding_refuses_what_the_library_cannot_see(zf):
    """Shapes, dtypes and devices of tensors: checked before any address is taken."""
    x, w = torch.zeros(4, 64), torch.zeros(64)
    with pytest.raises(ValueError, match="not on the current GPU"):
        zf.layer_norm(zf.NORM_RMS, x, w, None, 1e-5, torch.empty_like(x), None, torch.empty(4), stream=0)
    with pytest.raises(ValueError, match="one-byte"):
        zf.act8(torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="2 scales"):
        zf.act8(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 3, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        zf.act8(torch.zeros(64, 4, dtype=torch.uint8).t(), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="overlap"):
        zf.act8(torch.zeros(64, dtype=torch.uint8).expand(4, 64), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="was expected"):
        zf._matrix("t", x, 4, 63)
    with pytest.raises(ValueError, match="contiguous"):
        zf._matrix("t", x.t(), 64, 4)
    with pytest.raises(ValueError, match="unsupported"):
        zf._matrix("t", x.double(), 4, 64)
    with pytest.raises(ValueError, match="contiguous"):
        zf._vector("t", torch.zeros(128)[::2], 64)
    with pytest.raises(ValueError, match="does not fit"):
        zf._vector("t", w, 64, zf.BF16)
    with pytest.raises(ValueError, match="int32 or int64"):
        zf._ids("t", torch.zeros(4))


def test_the_definition_of_a_checkpoint():
    """The definition that the GPU tests compare with, on numbers worked out by hand."""
    table = R.e4m3_table()
    assert len(table) == 127 and table[0] == 0 and table[1] == 2.0 ** -9 and table[8] == 2.0 ** -6
    assert table[126] == 448 and table[119] == 240 and bool((table[1:] > table[:-1]).all())
    x = torch.zeros(1, 64, dtype=torch.bfloat16)
    x[0, :4] = torch.tensor([448.0, -1.0, 0.0, 2.0 ** -10])  # k = 0; half a least step: to even, zero
    x[0, 32:35] = torch.tensor([450.0, 3 * 2.0 ** -10, float("inf")])  # k = 1; rounds up to one step
    codes, scales = R.keep(x)
    assert scales.tolist() == [[127, 128]]
    assert codes[0, :4].tolist() == [126, 128 + 56, 0, 0] and codes[0, 32:35].tolist() == [118, 1, 127]
    back = R.numbers(codes, scales)
    assert back[0, 0] == 448 and back[0, 1] == -1 and back[0, 32] == 448 and back[0, 33] == 2.0 ** -8
    top = torch.tensor([[65504.0, 61440.0]], dtype=torch.float16)
    assert R.numbers(*R.keep(top)).tolist() == [[61440.0, 61440.0]]
    most = torch.tensor([[3.3e38, 1.0]], dtype=torch.bfloat16)
    codes, scales = R.keep(most)
    assert scales.item() == 247 and codes[0, 0] == 119


def test_a_planted_mistake_is_seen():
    """The comparison refuses a value one rounding too far, and an infinity where a number belongs."""
    want = torch.tensor([1.0, 2.0], dtype=torch.float64)
    bound = R.rounded(want, 0.0, torch.bfloat16)
    R.assert_within(torch.tensor([1.0, 2.0]), want, bound)
    with pytest.raises(AssertionError):
        R.assert_within(torch.tensor([1.0, 2.0 + 2.0 ** -6]), want, bound)
    with pytest.raises(AssertionError):
        R.assert_within(torch.tensor([1.0, float("inf")]), want, bound)
