"""Paths of the activation operators that depend on a shape's plan, on the GPU,
against float64."""
import pytest

from test_gpu_gn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("n,s,c,groups", [(1100, 1, 4096, 1), (300, 3, 4096, 2), (150, 4, 2500, 1), (140, 2, 3001, 1),
                                          (3, 2, 4224, 2), (140, 5, 4096, 1)])
def test_fp32_groups_wider_than_2048_channels(n, s, c, groups, act):
    """A column of lanes of its own for each four channels: short samples whole in 1024 lanes, several
    of them a workgroup; five positions, and all of them where samples are few, in chunks."""
    Case(n, s, c, groups, "f32", act, seed=c + s).check_all()
