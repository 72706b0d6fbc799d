"""The cases of the tests of zf_weight_grad's largest tiles take them (no GPU needed)."""
import pytest

from tests import weight_grad_plan as plan


@pytest.mark.parametrize("rows,outs,ins", plan.LARGE)
def test_large_tiles_without_splits(rows, outs, ins):
    assert plan.chosen(rows, outs, ins) == ("big", 1)
    assert outs % 8 == 0 and ins % 16 == 0, "whole pieces"
    assert rows % 32 and outs % 256 and ins % 256, "ends inside a stage and a tile"


def test_the_plan_is_the_librarys():
    """Where no form splits the tokens the library asks for no workspace; with splits, for those at least."""
    from fsdp_sharded_mixed_amd import zf
    for rows, outs, ins in plan.LARGE + [(6200, 2056, 2064), (16384, 256, 1024), (333, 776, 1008), (40, 2056, 2320)]:
        form, splits = plan.chosen(rows, outs, ins)
        need = zf.weight_grad_bytes(rows, outs, ins)
        assert need >= (splits * outs * ins * 4 if splits > 1 else 0)
        if (rows, outs, ins) in plan.LARGE:
            assert need == 0
    assert plan.chosen(6200, 2056, 2064) == ("big", 3) and plan.chosen(16384, 256, 1024) == ("little", 8)
    assert plan.chosen(333, 777, 1000, False) == ("little", 1) and plan.chosen(40, 2056, 2320) == ("middle", 1)
