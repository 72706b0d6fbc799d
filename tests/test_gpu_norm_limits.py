"""Norms of rows whose squares no binary32 number holds, and of rows without variance and eps = 0, as the header says."""
import pytest
import torch

from tests import rank_ops as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def zf():
    from fsdp_sharded_mixed_amd import zf as Z
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return Z


@pytest.mark.parametrize("kind", R.KINDS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [40, 300, 2048, 2050, 17000])
def test_rows(zf, kind, dtype, cols):
    g = R.generator(cols)
    x = R.normal(g, 7, cols)
    x[1] = torch.where(x[1] < 0, -2.0 ** 65, 2.0 ** 65)  # squares of 2^130
    x[3] = 0.0
    x[4] *= 2.0 ** 55  # squares within binary32
    x = x.to(dtype)
    w = torch.ones(cols, dtype=dtype, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(7, device="cuda")
    mean = torch.empty(7, device="cuda") if kind == "layer" else None
    k = zf.NORM_LAYER if kind == "layer" else zf.NORM_RMS
    for eps in (0.0, 1e-50, 1e-5):
        zf.layer_norm(k, x, w, None, eps, y, mean, rstd)
        assert float(rstd[1]) == 0 and bool((y[1] == 0).all())
        if eps < 1e-45:  # no binary32 number above zero
            assert bool(rstd[3].isinf() and y[3].isnan().all())
        else:
            assert bool((y[3] == 0).all())
        v = x.double() - (x.double().mean(1, keepdim=True) if kind == "layer" else 0)
        for i in (0, 2, 4, 5, 6):
            want = v[i] * (v[i].square().mean() + eps).rsqrt()
            # the mean's chain of additions, then the squares' and five roundings, for rows of unit deviation
            R.assert_within(y[i], want, R.rounded(want, (want.abs() + 1) * (80 + cols // 256 + 8) * 2 * R.U32, dtype), str(i))
