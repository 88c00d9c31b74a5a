"""The group norm and its gradients against the formulas in 64 bits.

u = 2^-24.  A mean or a sum of squares goes through at most `pixels` additions
in a thread (far fewer where a sample is shared) and some 40 in trees: K = (64 +
pixels / 16) u of the sum of magnitudes, with pixels of the test's size.  xh is
off by what the mean's error and its own subtraction leave, K rstd (|x| +
|mean|), and by rstd's, K |xh|.  silu's slope is at most 1.1 and its second
derivative at most 0.5.  bf16 results add half a step, 2^-8."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def f64(t):
    return t.detach().double().cpu().numpy()


def make(batch, pixels, channels, x="f32", y="f32", seed=0, mean=0.3, spread=1.0, w=True, b=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*s):
        return torch.randn(s, generator=g, device="cuda")
    return dict(x=(spread * rn(batch, pixels, channels) * (0.5 + torch.rand(channels, generator=g, device="cuda")) +
                   mean * (1 + 0.1 * rn(channels))).to(dt(x)),
                dy=rn(batch, pixels, channels).to(dt(y)), w=1 + 0.2 * rn(channels) if w else None,
                b=0.2 * rn(channels) if b else None)


def grouped(a, groups):
    return a.reshape(a.shape[0], a.shape[1], groups, -1)


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0), (z > 0).astype(float)
    if name == "silu":
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-z))
        return z * s, s + z * s * (1 - s)
    return z, np.ones_like(z)


def parts(a, groups, eps, mean=None, rstd=None):
    """x, mean, rstd, xh, w, b as [batch, pixels, groups, size], and xh's bound."""
    x = grouped(f64(a["x"]), groups)
    size = x.shape[3]
    K = (64 + x.shape[1] / 16) * U
    if mean is None:
        mean = x.mean((1, 3), keepdims=True)
        rstd = 1 / np.sqrt(((x - mean) ** 2).mean((1, 3), keepdims=True) + eps)
    else:
        mean, rstd = f64(mean)[:, None, :, None], f64(rstd)[:, None, :, None]
    w = f64(a["w"]).reshape(groups, size) if a["w"] is not None else np.ones((groups, size))
    b = f64(a["b"]).reshape(groups, size) if a["b"] is not None else np.zeros((groups, size))
    xh = (x - mean) * rstd
    return x, mean, rstd, xh, w, b, K, K * (rstd * (np.abs(x) + np.abs(mean)) + np.abs(xh))


def near(got, ref, tol, what):
    err = np.abs(f64(got).reshape(ref.shape) - ref)
    assert np.all(err <= tol + 1e-37), f"{what}: error {np.nanmax(err):.3e}, over its bound by {np.nanmax(err - tol):.3e}"


def forward(amd, a, groups, activation, eps=1e-5, y="f32", x=None):
    x = a["x"] if x is None else x
    got, mean, rstd = amd.group_norm(x, groups, a["w"], a["b"], eps=eps, activation=activation, y_dtype=dt(y))
    X, M, R, xh, w, b, K, txh = parts(a, groups, eps)
    z = xh * w + b
    ref, _ = act(z, activation)
    tz = txh * np.abs(w) + 2 * U * (np.abs(xh * w) + np.abs(b))
    tol = 1.1 * tz + 8 * U * np.abs(ref) * (1 + np.abs(z))
    near(mean, M[:, 0, :, 0], (K * np.abs(X).mean((1, 3), keepdims=True))[:, 0, :, 0], "mean")
    near(rstd, R[:, 0, :, 0], K * (R * (1 + R ** 2 * K * (X ** 2).mean((1, 3), keepdims=True)))[:, 0, :, 0], "rstd")
    assert got.dtype == dt(y) and got.shape == x.shape
    near(got, ref, tol + HALF[y] * (np.abs(ref) + tol), "y")
    return got, mean, rstd


def backward(amd, a, groups, activation, mean, rstd, x="f32"):
    import torch
    dx, dw, db = amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], mean, rstd, activation=activation)
    X, M, R, xh, w, b, _, _ = parts(a, groups, 0, mean, rstd)
    batch, pixels = X.shape[:2]
    K = (64 + pixels / 16) * U
    txh = 3 * U * np.abs(xh) + U * R * 0                                  # its inputs are given: three roundings
    z = xh * w + b
    up = grouped(f64(a["dy"]), groups)
    _, slope = act(z, activation)
    dz = up * slope
    tz = txh * np.abs(w) + 2 * U * (np.abs(xh * w) + np.abs(b))
    tdz = np.abs(up) * (0.5 * tz + 8 * U * (1 + np.abs(z))) * (activation == "silu") + U * np.abs(dz)
    t = dz * w

    def avg(v):
        return v.mean((1, 3), keepdims=True)
    ref = R * (t - avg(t) - xh * avg(t * xh))
    tt = tdz * np.abs(w) + U * np.abs(t)
    tol = R * (tt + avg(tt) + K * avg(np.abs(t)) + np.abs(xh) * (avg(tt * np.abs(xh) + np.abs(t) * txh) +
               K * avg(np.abs(t * xh))) + txh * np.abs(avg(t * xh))) + 8 * U * R * (
               np.abs(t) + np.abs(avg(t)) + np.abs(xh * avg(t * xh)))
    near(dx, ref, tol + HALF[x] * (np.abs(ref) + tol), "dx")
    assert dx.dtype == a["x"].dtype
    n = K + batch * U
    sums = ((dw, a["w"], dz * xh, tdz * np.abs(xh) + np.abs(dz) * txh + U * np.abs(dz * xh)), (db, a["b"], dz, tdz))
    for got, given, terms, each in sums:
        if given is None:
            assert got is None
        else:
            near(got, terms.sum((0, 1)).reshape(-1), (each + n * np.abs(terms)).sum((0, 1)).reshape(-1), "dw or db")
    again = amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], mean, rstd, activation=activation)
    assert all(p is q or torch.equal(p, q) for p, q in zip((dx, dw, db), again))


def both(amd, a, groups, activation, eps=1e-5, x="f32", y="f32"):
    _, mean, rstd = forward(amd, a, groups, activation, eps, y)
    backward(amd, a, groups, activation, mean, rstd, x)


SHAPES = [(1, 1, 8, 2), (2, 1, 1, 1), (3, 7, 6, 3), (2, 64, 64, 8), (1, 1000, 96, 8), (5, 33, 40, 5), (2, 323, 100, 4),
          (2, 300, 512, 32), (1, 50, 2048, 1), (2, 40, 1000, 1000), (300, 1, 64, 4), (70, 5, 24, 24), (1, 4099, 12, 2)]


@pytest.mark.parametrize("batch,pixels,channels,groups", SHAPES)
@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("activation", ["none", "relu", "silu"])
def test_group_norm(amd, batch, pixels, channels, groups, x, y, activation):
    both(amd, make(batch, pixels, channels, x, y, seed=pixels + channels), groups, activation, x=x, y=y)


# samples that fill more and more of the machine: one block's share, several, all
@pytest.mark.parametrize("pixels,channels,groups", [(3000, 64, 8), (16384, 32, 4), (16384, 64, 1), (66000, 16, 2),
                                                    (9001, 48, 3), (300, 4096, 2), (20000, 7, 1), (2500, 1536, 1)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_large_samples(amd, pixels, channels, groups, x):
    both(amd, make(2, pixels, channels, x, x, seed=channels), groups, "silu", x=x, y=x)


# tensors of which only a part is under way at once: results far behind the statistics, groups of many tiles
@pytest.mark.parametrize("batch,pixels,channels,groups", [(6, 9000, 256, 32), (3, 5000, 1500, 1), (2, 9000, 1024, 2)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_large_batches(amd, batch, pixels, channels, groups, x):
    both(amd, make(batch, pixels, channels, x, x, seed=channels), groups, "silu", x=x, y=x)


@pytest.mark.parametrize("way", ["forward", "backward"])
def test_wait_that_gives_up_is_reported(amd, way):
    """With no patience the blocks of results stop waiting for statistics: the
    call ends and says so, and the next one is right."""
    import torch
    a = make(4, 20000, 64)
    want = amd.group_norm(a["x"], 8, a["w"], a["b"])
    back = amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], *want[1:])
    amd.amsim_device_errors()
    try:
        amd.amsim_set_flag_wait_limit(0)
        for _ in range(5):
            if way == "forward":
                amd.group_norm(a["x"], 8, a["w"], a["b"])
            else:
                amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], *want[1:])
        rc, bits = amd.amsim_device_errors()
    finally:
        amd.amsim_set_flag_wait_limit(2_000_000_000)
    assert rc == amd.AMSIM_ETIMEOUT and bits == amd.AMSIM_WAIT_PARTIAL
    assert all(torch.equal(p, q) for p, q in zip(amd.group_norm(a["x"], 8, a["w"], a["b"]), want))
    assert all(torch.equal(p, q) for p, q in zip(
        amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], *want[1:]), back))
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)


@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
def test_without_weights(amd, w, b):
    both(amd, make(2, 77, 24, w=w, b=b), 3, "silu")


@pytest.mark.parametrize("pixels", [60, 5000])
@pytest.mark.parametrize("mean,spread", [(1000.0, 1.0), (-3e4, 0.1), (1e-20, 1e-20), (0.0, 1e15), (5.0, 0.0)])
def test_means_far_from_zero(amd, pixels, mean, spread):
    """Groups whose mean is large against their deviation, or that are constant."""
    a = make(2, pixels, 24, seed=3, mean=mean, spread=spread)
    _, m, r = forward(amd, a, 4, "none")
    backward(amd, a, 4, "none", m, r)


def test_relu_at_its_edge(amd):
    """z that is exactly or almost zero: the gradient's sign is that of the exact z."""
    import torch
    a = make(1, 512, 16, seed=5)
    _, mean, rstd = amd.group_norm(a["x"], 2, a["w"], a["b"])
    X, M, R, xh, w, b, _, _ = parts(a, 2, 0, mean, rstd)
    # shift b channel by channel so that pixel 100's z falls within a rounding of zero
    a["b"] = torch.from_numpy((-(xh * w)[0, 100]).reshape(-1)).float().cuda()
    backward(amd, a, 2, "relu", mean, rstd)
    z = xh * w + f64(a["b"]).reshape(2, 8)
    assert (np.abs(z[0, 100]) < 1e-6).all()
    dx = amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], mean, rstd, activation="relu")
    db = (grouped(f64(a["dy"]), 2) * (z > 0)).sum((0, 1)).reshape(-1)
    assert np.allclose(f64(dx[2]), db, rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("pixels", [40, 30000])
def test_non_finite_group(amd, value, pixels):
    import torch
    a = make(3, pixels, 16)
    clean, _, _ = amd.group_norm(a["x"], 2, a["w"], a["b"], activation="relu")
    a["x"][1, 17, 3] = float(value)
    y, mean, rstd = amd.group_norm(a["x"], 2, a["w"], a["b"], activation="relu")
    assert bool(torch.isnan(y[1, :, :8]).all())
    assert torch.equal(y[0], clean[0]) and torch.equal(y[2], clean[2]) and torch.equal(y[1, :, 8:], clean[1, :, 8:])
    dx, dw, db = amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], mean, rstd, activation="none")
    assert bool(torch.isnan(dx[1, :, :8]).all()) and bool(torch.isfinite(dx[[0, 2]]).all())
    assert bool(torch.isnan(dw[:8]).all()) and bool(torch.isfinite(dw[8:]).all())


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("pixels", [37, 9000])
@pytest.mark.parametrize("ld,off", [(32, 0), (24, 3), (27, 0), (40, 8), (25, 1)])
def test_strides_and_alignment(amd, x, y, pixels, ld, off):
    """A slice of wider pixels, tensors off 16 bytes: within the same bounds,
    nothing beside the slice written, in place."""
    import torch
    a = make(2, pixels, 24, x, y, seed=off)
    want = amd.group_norm(a["x"], 3, a["w"], a["b"], activation="silu", y_dtype=dt(y))

    def place(t, dtype):
        buf = torch.full((2 * pixels * ld + 64,), 7.0, dtype=dtype, device="cuda")
        v = buf[off:off + 2 * pixels * ld].view(2, pixels, ld)[..., :24]
        if t is not None:
            v.copy_(t)
        return buf, v
    (_, xv), (ybuf, yv), (_, dyv), (dxbuf, dxv) = (place(a["x"], dt(x)), place(None, dt(y)), place(a["dy"], dt(y)),
                                                   place(None, dt(x)))
    got, mean, rstd = forward(amd, a, 3, "silu", y=y, x=xv)
    types = dict(f32=amd.AMSIM_F32, bf16=amd.AMSIM_BF16)
    d = amd.GroupNormDesc(batch=2, pixels=pixels, ldx=ld, ldy=ld, lddx=ld, channels=24, groups=3, x_type=types[x],
                          y_type=types[y], activation=amd.AMSIM_ACT_SILU, eps=1e-5)
    ws = amd.workspace(max(amd.amsim_group_norm_workspace_size(d, i) for i in (0, 1)))
    amd.amsim_group_norm_fwd(d, xv, a["w"], a["b"], yv, mean, rstd, ws)
    assert torch.equal(yv, got)
    assert int((ybuf == 7).sum()) >= ybuf.numel() - 2 * pixels * 24
    rest = ybuf[off:off + 2 * pixels * ld].view(2, pixels, ld)[..., 24:]
    assert bool((rest == 7).all()) and bool((ybuf[:off] == 7).all()) and bool((ybuf[off + 2 * pixels * ld:] == 7).all())
    dx, dw, db = torch.empty_like(a["x"]), torch.empty_like(a["w"]), torch.empty_like(a["b"])
    amd.amsim_group_norm_bwd(d, dyv, xv, a["w"], a["b"], mean, rstd, dxv, dw, db, ws)
    ref = amd.group_norm_backward(dyv, xv, a["w"], a["b"], mean, rstd, activation="silu")
    assert torch.equal(dxv, ref[0]) and torch.equal(dw, ref[1]) and torch.equal(db, ref[2])
    if x == y:
        amd.amsim_group_norm_bwd(d, dyv, xv, a["w"], a["b"], mean, rstd, dyv, None, None, ws)
        assert torch.equal(dyv, dxv)
        amd.amsim_group_norm_fwd(d, xv, a["w"], a["b"], xv, mean, rstd, ws)
        assert torch.equal(xv, yv)


def test_empty(amd):
    import torch
    w = torch.ones(8, device="cuda")
    for shape in ((0, 5, 8), (2, 0, 8)):
        x = torch.zeros(shape, device="cuda")
        y, mean, rstd = amd.group_norm(x, 2, w, w, eps=0.25)
        assert y.shape == x.shape and not mean.any() and bool((rstd == 2).all())
        dx, dw, db = amd.group_norm_backward(x, x, w, w, mean, rstd)
        assert dx.shape == x.shape and not dw.any() and not db.any()


def test_shapes_of_images(amd):
    """NHWC and any other number of dimensions between batch and channels."""
    import torch
    a = make(2, 60, 12)
    want = amd.group_norm(a["x"], 4, a["w"], a["b"])
    for shape in ((2, 6, 10, 12), (2, 3, 4, 5, 12)):
        got = amd.group_norm(a["x"].view(shape), 4, a["w"], a["b"])
        assert got[0].shape == shape and torch.equal(got[0].view(2, 60, 12), want[0]) and torch.equal(got[1], want[1])
        back = amd.group_norm_backward(a["dy"].view(shape), a["x"].view(shape), a["w"], a["b"], *got[1:])
        assert back[0].shape == shape
    flat = amd.group_norm(a["x"][:, 0], 4, a["w"], a["b"])                # [batch, channels], batch strided
    assert torch.equal(flat[0], amd.group_norm(a["x"][:, :1].contiguous(), 4, a["w"], a["b"])[0][:, 0])


def test_refusals(amd):
    import torch
    a = make(2, 6, 12)
    x, w, b = a["x"], a["w"], a["b"]
    _, mean, rstd = amd.group_norm(x, 4, w, b)
    for args in ((x, 5, w, b), (x, 0, w, b), (x, 4, w[:11], b), (x[0, 0], 4, w, b), (x.transpose(1, 2), 2, None, None),
                 (x[..., ::2], 2, None, None), (x[:, ::2][:, :2], 4, w, b)):
        with pytest.raises(ValueError):
            amd.group_norm(*args)
    for args in ((x.half(), 4, w, b), (x, 4, w.double(), b), (x, 4, w, b.bfloat16())):
        with pytest.raises(TypeError):
            amd.group_norm(*args)
    with pytest.raises(ValueError):
        amd.group_norm(x, 4, w, b, activation="tanh")
    with pytest.raises(amd.AmsimError):
        amd.group_norm(x, 4, w, b, eps=-1.0)
    with pytest.raises(ValueError):
        amd.group_norm_backward(a["dy"][:1], x, w, b, mean, rstd)
    with pytest.raises(ValueError):
        amd.group_norm_backward(a["dy"], x, w, b, mean, rstd[:1])
    with pytest.raises(TypeError):
        amd.group_norm_backward(a["dy"], x, w, b, mean.double(), rstd)


def test_gradient_by_differences(amd):
    """dx, dw and db of a weighted sum of y against central differences.  With
    steps of h = 2^-5 about values of 1 a third derivative leaves about h^2 and
    the outputs' 2^-17 in 160 places 160 * 2^-17 / h / 8 (their signs differ)."""
    import torch
    a = make(1, 20, 8, seed=11)

    def value():
        return float((amd.group_norm(a["x"], 2, a["w"], a["b"], activation="silu")[0].double() * a["dy"]).sum())
    _, mean, rstd = amd.group_norm(a["x"], 2, a["w"], a["b"], activation="silu")
    grads = amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], mean, rstd, activation="silu")
    h, size = 2.0 ** -5, float(a["dy"].abs().max())
    for x, got in zip((a["x"], a["w"], a["b"]), grads):
        flat = x.view(-1)
        for i in range(0, flat.numel(), 3):
            keep = float(flat[i])
            flat[i] = keep + h
            up = value()
            flat[i] = keep - h
            down = value()
            flat[i] = keep
            assert abs((up - down) / (2 * h) - float(got.reshape(-1)[i])) <= 5e-3 * size


def test_streams_and_graphs(amd):
    import torch
    a, c = make(8, 900, 64, seed=1), make(8, 900, 64, seed=2)

    def call(a):
        y, m, r = amd.group_norm(a["x"], 8, a["w"], a["b"], activation="silu")
        return (y, m, r, *amd.group_norm_backward(a["dy"], a["x"], a["w"], a["b"], m, r, activation="silu"))
    want = [call(a), call(c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        outs = []
        for st, v in zip(streams, (a, c)):
            with torch.cuda.stream(st):
                outs.append(call(v))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for o, w in zip(outs, want) for p, q in zip(o, w))
    fixed = {k: v.clone() for k, v in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(fixed)
    for v, w in zip((a, c), want):
        for k in fixed:
            fixed[k].copy_(v[k])
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(out, w))
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)
