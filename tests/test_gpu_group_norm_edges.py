"""The group norm where a thread holds a whole group and where groups are
constant or far from zero.  u = 2^-24, bf16 results add half a step, 2^-8."""
import pytest

from test_gpu_group_norm import HALF, U, dt, f64, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("size", [1, 2, 4, 8, 12])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("pixels", [1, 2])
def test_non_finite_value_makes_its_small_group_nan(amd, x, y, size, value, pixels):
    """Wherever the value stands among the few of its group, and no other group sees it."""
    import torch
    a = make(3, pixels, 3 * size, x, y, seed=size)
    kw = dict(activation="relu", y_dtype=dt(y))
    clean, _, _ = amd.group_norm(a["x"], 3, a["w"], a["b"], **kw)
    for place in range(size):
        bad = a["x"].clone()
        bad[1, pixels - 1, size + place] = float(value)
        got, mean, rstd = amd.group_norm(bad, 3, a["w"], a["b"], **kw)
        group = got[1, :, size:2 * size]
        assert bool(torch.isnan(group).all()), f"place {place}: {group.tolist()}"
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[1, :, size:2 * size] = False
        assert torch.equal(got[rest], clean[rest])
        dx, _, _ = amd.group_norm_backward(a["dy"], bad, a["w"], a["b"], mean, rstd)
        assert bool(torch.isnan(dx[1, :, size:2 * size]).all()) and bool(torch.isfinite(dx[rest]).all())
