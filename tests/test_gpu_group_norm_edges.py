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


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("pixels,channels,groups", [(60, 24, 4), (5000, 24, 4), (900, 64, 8), (1, 16, 4), (300, 1000, 1)])
@pytest.mark.parametrize("activation", ["none", "relu", "silu"])
def test_group_of_one_value_gives_the_activation_of_b(amd, x, y, pixels, channels, groups, activation):
    """Its mean is that value and x - mean is zero, however large the value is
    against the square root of eps: what is left is the activation's own error
    (as the other tests count it) and a bf16 result's rounding.  For a value of
    up to four deviations (of 1 / sqrt(eps)) from zero a bf16 result may first
    take mean rstd w from b, and is off by u of both."""
    import torch
    a = make(5, pixels, channels, x, y, seed=channels)
    for i, value in enumerate((3000.0, -1000.0, 0.71875, 2.0 ** 60, 2.0 ** -9)):       # all of them bf16's
        a["x"][i] = value
    got, mean, rstd = amd.group_norm(a["x"], groups, a["w"], a["b"], activation=activation, y_dtype=dt(y))
    b = a["b"].double()
    ref = dict(none=b, relu=b.clamp(min=0), silu=b * torch.sigmoid(b))[activation]
    tol = (8 * U * ref.abs() * (1 + b.abs()) * (activation == "silu")).expand(5, 1, channels).clone()
    tol[4] += 1.1 * U * (b.abs() + 4 * a["w"].double().abs()) * (y == "bf16")
    assert bool(((got.double() - ref).abs() <= tol + HALF[y] * (ref.abs() + tol)).all())
    assert torch.equal(mean, a["x"][:, 0, :1].float().expand(5, groups))
    db = amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], mean, rstd, activation="relu")[2]
    up = a["dy"].double() * (b > 0)                                       # relu's sign is that of the same z
    assert bool(((db.double() - up.sum((0, 1))).abs() <= 600 * U * up.abs().sum((0, 1))).all())


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("pixels", [60, 5000])
@pytest.mark.parametrize("mean,spread", [(1000.0, 1.0), (300.0, 0.1), (-3e4, 30.0), (0.5, 1.0)])
def test_groups_far_from_zero(amd, y, pixels, mean, spread):
    """All of a group about one mean.  A thread's mean and each joining of two
    means rounds once, u |mean|; from a thread's values to a sample's statistics
    there are at most 20 in a row here, so the mean is within M = 21 u |mean| and
    what the sums about a first value and the joins lose, L = 256 u deviations.  A sum of squares
    is within 3 (64 + 8) u of itself (values about a first one some deviations
    away; a thread has at most 48) and, as each of 20 levels joins means that are
    off by D = 2 M from another, 2 (D / s) sqrt(10) + 10 (D / s)^2 more; rstd is
    off by half of that.  x - mean carries the mean's error and one rounding; the
    rest is as in the other tests."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    a = make(2, pixels, 24, y=y, seed=3)
    a["x"] = mean + spread * torch.randn((2, pixels, 24), generator=g, device="cuda")
    got, m, r = amd.group_norm(a["x"], 4, a["w"], a["b"], y_dtype=dt(y))
    X = f64(a["x"]).reshape(2, pixels, 4, 6)
    M = X.mean((1, 3))
    s = X.std((1, 3))
    R = (s ** 2 + 1e-5) ** -0.5
    off = 21 * U * abs(M) + 256 * U * s
    assert (abs(f64(m) - M) <= off).all()
    D = 2 * off / s
    tr = (3 * 72 * U + 2 * D * 10 ** 0.5 + 10 * D ** 2) / 2 + 4 * U
    assert (tr < 0.03).all() and (abs(f64(r) / R - 1) <= tr).all()
    M, R, off, tr = (v[:, None, :, None] for v in (M, R, off, tr))
    w, b = (f64(a[k]).reshape(4, 6) for k in "wb")
    xw = (X - M) * R * w
    ref = xw + b
    tol = R * abs(w) * off * (1 + tr) + abs(xw) * (tr + 4 * U) + 2 * U * (abs(xw) + abs(b))
    assert (abs(f64(got).reshape(ref.shape) - ref) <= tol + HALF[y] * (abs(ref) + tol)).all()


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("pixels", [60, 5000])
def test_groups_near_and_far_from_zero_side_by_side(amd, x, y, pixels):
    """Groups of eight channels whose threads share warps, at -2000, 0, 3, 100
    and a constant 500.  From mean and rstd as they are: the subtraction, the
    product with rstd (or of rstd and w) and the sum with b each round once, 4 u
    |xh w| and 2 u of the terms; a bf16 result whose mean is up to four deviations
    from zero may first take mean rstd w from b, u 4 |w| more.  bf16 adds half a step."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(10)
    a = make(2, pixels, 40, y=y, seed=4)
    at = torch.tensor([-2000.0, 0.0, 3.0, 100.0, 500.0], device="cuda").repeat_interleave(8)
    wide = torch.tensor([1.0, 1.0, 1.0, 1.0, 0.0], device="cuda").repeat_interleave(8)
    a["x"] = (at + wide * torch.randn((2, pixels, 40), generator=g, device="cuda")).to(dt(x))
    got, m, r = amd.group_norm(a["x"], 5, a["w"], a["b"], y_dtype=dt(y))
    M, R = f64(m)[:, None, :, None], f64(r)[:, None, :, None]
    w, b = (f64(a[k]).reshape(5, 8) for k in "wb")
    xh = (f64(a["x"]).reshape(2, pixels, 5, 8) - M) * R
    ref = xh * w + b
    near = (abs(M) * R <= 4.001) * (y == "bf16")
    tol = abs(w) * U * (4 * abs(xh) + 4 * near) + 2 * U * (abs(xh * w) + abs(b))
    assert (abs(f64(got).reshape(ref.shape) - ref) <= tol + HALF[y] * (abs(ref) + tol)).all()
    assert not (ref - b)[:, :, 4].any()
