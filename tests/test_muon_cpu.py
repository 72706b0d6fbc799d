"""Argument checks of the Muon calls (no GPU needed): every call here returns
before the HIP runtime is touched, and leaves nothing enqueued.  Device
addresses are made-up numbers that no kernel sees."""
import ctypes as C

import pytest

from fsdp_sharded_mixed_amd import workloads as W

BASE = 1 << 20


@pytest.fixture(scope="module")
def zf():
    from fsdp_sharded_mixed_amd import zf as Z
    return Z


def status(zf, fn, *args):
    with pytest.raises(zf.ZfError) as e:
        fn(*args)
    return zf.STATUS[e.value.status]


def batch(zf, shapes, src=None, dst=None, **kw):
    arr = (zf.Matrix * len(shapes))()
    for i, (r, c) in enumerate(shapes):
        arr[i] = zf.Matrix(kw.get("src_ptr", BASE), kw.get("dst_ptr", 2 * BASE), r, c,
                           kw.get("src_stride", c), kw.get("dst_stride", c))
    return zf.OrthoBatch(arr, kw.get("count", len(shapes)), src or zf.F32, dst or zf.BF16, None, ())


def call(zf, b, ns=None, ws=3 * BASE, size=1 << 40):
    zf.orthogonalize(b, ws, ns=ns, stream=0, workspace_size=size)


def test_empty_batch_is_a_no_op(zf):
    b = batch(zf, [])
    assert zf.orthogonalize_bytes(b) == 0
    call(zf, b, ws=None, size=0)


@pytest.mark.parametrize("shape", [(0, 4), (4, 0), (-1, 4)])
def test_sides_below_one(zf, shape):
    assert status(zf, call, zf, batch(zf, [shape])) == "ZF_EINVAL"
    assert status(zf, zf.orthogonalize_bytes, batch(zf, [shape])) == "ZF_EINVAL"


@pytest.mark.parametrize("kw,want", [
    ({"src_ptr": None}, "ZF_EINVAL"), ({"dst_ptr": None}, "ZF_EINVAL"),
    ({"src_stride": 7}, "ZF_EINVAL"), ({"dst_stride": 7}, "ZF_EINVAL"),
    ({"src_ptr": BASE + 2}, "ZF_EALIGN"), ({"dst_ptr": BASE + 1}, "ZF_EALIGN"),
    ({"src": 9}, "ZF_EDTYPE"), ({"dst": 9}, "ZF_EDTYPE"), ({"count": -1}, "ZF_EINVAL")])
def test_bad_batches(zf, kw, want):
    assert status(zf, call, zf, batch(zf, [(8, 8)], **kw)) == want


@pytest.mark.parametrize("places,want", [
    ([(1, 2), (3, 2)], "ZF_EINVAL"),   # two results in one place
    ([(1, 2), (1, 4)], "ZF_ESIZE"),    # one matrix twice: fine
    ([(1, 1), (2, 2)], "ZF_ESIZE"),    # each in place: fine
    ([(1, 2), (2, 3)], "ZF_EINVAL"),   # a result where another matrix lies
    ([(1, 1), (1, 1)], "ZF_EINVAL"), ([(1, 1), (1, 2)], "ZF_EINVAL")])
def test_results_in_other_matrices_places(zf, places, want):
    b = batch(zf, [(8, 8)] * 2)
    for m, (src, dst) in zip(b.mats, places):
        m.src, m.dst = src * BASE, dst * BASE
    # those that pass are refused for their workspace, the last check
    assert status(zf, call, zf, b, None, 9 * BASE, 0) == want


def test_buffers_elsewhere(zf, monkeypatch):
    import torch
    b = batch(zf, [(8, 8)])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for where in ("cpu", "cuda:1"):
        b.device = torch.device(where)
        with pytest.raises(ValueError, match="current GPU"):
            call(zf, b)
    b.device = torch.device("cuda:0")
    assert status(zf, call, zf, b, None, 3 * BASE, 0) == "ZF_ESIZE"
    with pytest.raises(ValueError, match="current GPU"):
        call(zf, b, ws=torch.zeros(16))
    with pytest.raises(ValueError, match="on a GPU"):
        zf.ortho_batch([torch.zeros(4, 6)], [torch.zeros(4, 6)])
    with pytest.raises(ValueError, match="current GPU"):
        step(zf, master=torch.zeros(1 << 18))


def test_strides_of_single_rows_are_ignored(zf):
    # refused for its workspace, the last check: the stride has passed
    b = batch(zf, [(1, 8)], src_stride=1, dst_stride=1)
    assert status(zf, call, zf, b, None, 3 * BASE, 0) == "ZF_ESIZE"


def test_sides_above_the_limit(zf):
    assert status(zf, call, zf, batch(zf, [(1, (1 << 20) + 1)])) == "ZF_ESIZE"


def test_workspace_checks(zf):
    b = batch(zf, [(8, 8)])
    need = zf.orthogonalize_bytes(b)
    assert need > 0
    assert status(zf, call, zf, b, None, 3 * BASE, need - 1) == "ZF_ESIZE"
    assert status(zf, call, zf, b, None, None, need) == "ZF_EINVAL"
    assert status(zf, call, zf, b, None, 3 * BASE + 8, need) == "ZF_EALIGN"


@pytest.mark.parametrize("kw", [{"steps": 0}, {"steps": 33}, {"products": 2}, {"products": -1},
                                {"a": float("nan")}, {"b": float("inf")}, {"c": float("nan")},
                                {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}])
def test_iteration_parameters(zf, kw):
    assert status(zf, call, zf, batch(zf, [(8, 8)]), zf.ns_params(**kw)) == "ZF_EINVAL"
    assert status(zf, zf.orthogonalize_bytes, batch(zf, [(8, 8)]), zf.ns_params(**kw)) == "ZF_EINVAL"


def test_more_products_need_more_workspace(zf):
    b = batch(zf, [(512, 512)])
    assert zf.orthogonalize_bytes(b, zf.ns_params(products=3)) > zf.orthogonalize_bytes(b)
    f32 = batch(zf, [(512, 512)], dst=zf.F32)
    assert zf.orthogonalize_bytes(f32) == zf.orthogonalize_bytes(b, zf.ns_params(products=3))


def test_ortho_batch_refuses(zf):
    import torch
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="as many outs"):
        zf.ortho_batch([x], [])
    with pytest.raises(ValueError, match="2-D"):
        zf.ortho_batch([x[0]], [x[0]])
    with pytest.raises(ValueError, match="shaped as"):
        zf.ortho_batch([x], [x[:2]])
    with pytest.raises(ValueError, match="contiguous"):
        zf.ortho_batch([x.t()], [x.t()])
    with pytest.raises(ValueError, match="overlap"):
        zf.ortho_batch([x[:1].expand(4, 6)], [x])
    with pytest.raises(ValueError, match="one dtype"):
        zf.ortho_batch([x, x.half()], [x, x])
    with pytest.raises(ValueError, match="dtype"):
        zf.ortho_batch([x.double()], [x.double()])


# the first matrix is more than a round of blocks, the second is held in shared memory
SEGS = [(1100 * 1300, 0, 0, 1100), (6, 0, 0, 0), (35, 1, 0, 7), (35, 1, 0, 0)]


def plan(zf, layout=W.PER_UNIT, n=3):
    return zf.plan_flat(SEGS, n, layout, 2)


@pytest.mark.parametrize("layout", [W.GLOBAL_FLAT, W.PER_UNIT, W.PER_PARAM_DIM0])
def test_muon_plan(zf, layout):
    m = zf.muon_plan(plan(zf, layout), [2, 0])
    assert zf.muon_workspace_bytes(m) > 0
    assert zf.muon_workspace_bytes(m, zf.ns_params(products=3)) > zf.muon_workspace_bytes(m)
    assert status(zf, zf.muon_workspace_bytes, m, zf.ns_params(steps=0)) == "ZF_EINVAL"


@pytest.mark.parametrize("segments", [[], [4], [-1], [0, 0], [1], [0, 3], [0, 1, 2, 3, 0]])
def test_muon_plan_refuses(zf, segments):
    # none, out of range, twice, vectors
    assert status(zf, zf.muon_plan, plan(zf), segments) == "ZF_EINVAL"


def test_muon_plan_refuses_rows_that_do_not_divide(zf):
    p = zf.plan_flat([(35, 0, 0, 6)], 2, W.GLOBAL_FLAT, 2)
    assert status(zf, zf.muon_plan, p, [0]) == "ZF_EINVAL"


def test_few_thin_blocks_take_three_products(zf):
    """Up to 256 blocks of 64 x 64 beside the matrices held in shared memory,
    one of them thin."""
    exact = zf.ns_params(products=3)
    for rows, cols, few in ((1024, 1024, False), (32, 16384, True), (32, 16385, False),
                            (33, 4000, False), (1293, 4, True)):
        m = zf.muon_plan(zf.plan_flat([(rows * cols, 0, 0, rows), (35, 0, 0, 7)], 2,
                                      W.GLOBAL_FLAT, 2), [0, 1])
        assert (zf.muon_workspace_bytes(m) == zf.muon_workspace_bytes(m, exact)) == few


def test_muon_plan_outlives_its_plan(zf):
    p = plan(zf)
    m = zf.muon_plan(p, [0])
    del p
    assert zf.muon_workspace_bytes(m) > 0


def test_muon_null_pointers(zf):
    out = C.c_void_p()
    seg = (C.c_int64 * 1)(0)
    p = plan(zf)
    assert zf.lib.zf_muon_plan(None, seg, 1, C.byref(out)) == -1
    assert zf.lib.zf_muon_plan(p.handle, None, 1, C.byref(out)) == -1
    assert zf.lib.zf_muon_plan(p.handle, seg, 1, None) == -1
    assert zf.lib.zf_muon_workspace_bytes(None, None) == -1
    zf.lib.zf_muon_free(None)


def step(zf, **kw):
    layout = kw.pop("layout", W.PER_UNIT)
    p = plan(zf, layout)
    m = zf.muon_plan(p, [0, 2])
    mhp = kw.pop("mhp", zf.muon_hparams(1e-3))
    size = kw.pop("size", zf.muon_workspace_bytes(m) if mhp.ns.steps else 1 << 30)
    args = dict(grad_dtype=zf.BF16, param_dtype=zf.BF16, grads=[BASE] * 3, master=2 * BASE,
                exp_avg=3 * BASE, exp_avg_sq=4 * BASE, params=5 * BASE, workspace=6 * BASE,
                state=7 * BASE, grad_shards=8 * BASE if layout == W.PER_PARAM_DIM0 else None,
                numel=p.psi_pad)
    args.update(kw)
    zf.muon_step(m, kw.get("hp", zf.hparams(1e-3)), mhp, args["grad_dtype"], args["param_dtype"],
                 args["grads"], args["master"], args["exp_avg"], args["exp_avg_sq"],
                 args["params"], args["workspace"], args["state"], stream=0,
                 grad_shards=args["grad_shards"], numel=args["numel"], workspace_size=size,
                 grads_reduced=args.get("grads_reduced", False))


@pytest.mark.parametrize("kw,want", [
    ({"master": None}, "ZF_EINVAL"), ({"exp_avg": None}, "ZF_EINVAL"),
    ({"exp_avg_sq": None}, "ZF_EINVAL"), ({"state": None}, "ZF_EINVAL"),
    ({"workspace": None}, "ZF_EINVAL"), ({"grads": None}, "ZF_EINVAL"),
    ({"grads": [BASE, None, BASE]}, "ZF_EINVAL"), ({"grads_reduced": True}, "ZF_EINVAL"),
    ({"layout": W.PER_PARAM_DIM0, "grad_shards": None}, "ZF_EINVAL"),
    ({"master": BASE + 4}, "ZF_EALIGN"), ({"params": BASE + 2}, "ZF_EALIGN"),
    ({"workspace": BASE + 8}, "ZF_EALIGN"), ({"grad_dtype": 3}, "ZF_EDTYPE"),
    ({"param_dtype": 3}, "ZF_EDTYPE"), ({"numel": 100}, "ZF_ESIZE"), ({"size": 1024}, "ZF_ESIZE")])
def test_muon_step_refuses(zf, kw, want):
    assert status(zf, lambda: step(zf, **kw)) == want


@pytest.mark.parametrize("kw", [{"momentum": 1.0}, {"momentum": -0.1},
                                {"momentum": float("nan")}, {"nesterov": 2}, {"scale_rule": 2}])
def test_muon_hparams_refused(zf, kw):
    assert status(zf, lambda: step(zf, mhp=zf.muon_hparams(1e-3, **kw))) == "ZF_EINVAL"


def test_muon_step_refuses_iteration_parameters(zf):
    bad = zf.muon_hparams(1e-3, ns=zf.ns_params(steps=0))
    assert status(zf, lambda: step(zf, mhp=bad)) == "ZF_EINVAL"


def test_muon_step_needs_the_workspace_of_its_products(zf):
    fine = zf.muon_hparams(1e-3, ns=zf.ns_params(products=3))
    assert status(zf, lambda: step(zf, mhp=fine)) == "ZF_ESIZE"


def test_muon_step_refuses_betas(zf):
    assert status(zf, lambda: step(zf, hp=zf.hparams(1e-3, beta1=1.0))) == "ZF_EINVAL"
