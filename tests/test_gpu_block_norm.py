"""The block norm against its formulas in 64 bits, elementwise, with bounds from
the fp32 arithmetic: a row's sum of squares goes through at most 16 + 10
sequential or tree additions per thread and row, so rstd is within 32 u of its
64-bit value (u = 2^-24), and each output adds a few roundings on top; K = 64 u
of the magnitudes that enter covers both.  Types of 16 bits add half an ulp of
the result (2^-8).  Column sums over R rows add R + 64 u of the sum of the
magnitudes."""
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
K = 64 * U
HALF = {"f32": U, "bf16": 2.0 ** -8}


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(rows, cols, x="f32", y="f32", n="f32", groups=1, post=True, pre=True, gate=True, seed=0, has_y=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*s):
        return torch.randn(s, generator=g, device="cuda")
    return dict(x=(2 * rn(rows, cols)).to(dt(x)), y=(1.3 * rn(rows, cols)).to(dt(y)) if has_y else None,
                w_post=1 + 0.1 * rn(cols) if post and has_y else None, w_pre=1 + 0.1 * rn(cols) if pre else None,
                gate=0.5 + 0.3 * rn(groups, cols) if gate and has_y else None, n_type=dt(n),
                dr=rn(rows, cols).to(dt(x)), dn=rn(rows, cols).to(dt(n)))


def rows_of_gate(a, rows):
    return np.repeat(a, rows // a.shape[0], 0)


def ref_fwd(a, alpha, eps):
    x = f64(a["x"])
    C = x.shape[1]
    size = np.abs(x)
    post = None
    if a["y"] is None:
        r = x
    else:
        u = f64(a["y"])
        if a["w_post"] is not None:
            post = 1 / np.sqrt((u * u).mean(1) + eps)
            u = u * post[:, None] * f64(a["w_post"])
        if a["gate"] is not None:
            u = u * rows_of_gate(f64(a["gate"]), x.shape[0])
        r = x + alpha * u
        size = size + np.abs(alpha * u)
    pre = 1 / np.sqrt((r * r).mean(1) + eps)
    w = f64(a["w_pre"]) if a["w_pre"] is not None else np.ones(C)
    return r, r * pre[:, None] * w, post, pre, size, size * pre[:, None] * np.abs(w)


def check(got, ref, tol, what):
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), f"{what}: error {err.max():.3e}, over its bound by {(err - tol).max():.3e}"


SHAPES = [(1, 1), (3, 7), (2, 8), (130, 64), (33, 1000), (5, 1013), (17, 4096), (4, 4100), (6, 8200), (3, 16384),
          (3, 16383)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("x,y,n", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"),
                                   ("bf16", "f32", "f32")])
def test_forward(amd, rows, cols, x, y, n):
    a = make(rows, cols, x, y, n, seed=rows + cols)
    r, nn, post, pre = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=0.5, eps=1e-5,
                                      n_dtype=a["n_type"])
    R, N, P, Q, sr, sn = ref_fwd(a, 0.5, 1e-5)
    assert r.dtype == a["x"].dtype and nn.dtype == a["n_type"]
    check(r, R, K * sr + HALF[x] * (1 + K) * np.abs(R), "r")
    # the norm of r moves with r's own error, at most K of its largest row magnitudes
    check(nn, N, 2 * K * sn + K * np.abs(N) + HALF[n] * (1 + K) * np.abs(N) + K * np.abs(N).max(), "n")
    check(post, P, K * P, "rstd_post")
    check(pre, Q, 2 * K * Q, "rstd_pre")


@pytest.mark.parametrize("has_y,post,pre,gate,groups", [
    (False, False, True, False, 1), (False, False, False, False, 1), (True, False, True, False, 1),
    (True, True, False, False, 1), (True, False, True, True, 4), (True, True, True, True, 12)])
def test_forward_without_parts(amd, has_y, post, pre, gate, groups):
    a = make(12, 72, "f32", "bf16", "f32", groups, post, pre, gate, seed=4, has_y=has_y)
    r, n, p, q = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=-2.0, eps=0.0,
                                n_dtype=a["n_type"])
    R, N, P, Q, sr, sn = ref_fwd(a, -2.0, 0.0)
    check(r, R, K * sr, "r")
    check(n, N, 4 * K * sn + K * np.abs(N).max(), "n")
    assert (p is None) == (not post)
    if not has_y:
        assert r is a["x"]


def ref_bwd(a, r, alpha, post, pre):
    """Gradients and, with them, the magnitudes that enter each."""
    y, dr, dn = f64(a["y"]), f64(a["dr"]), f64(a["dn"])
    rows, C = f64(r).shape
    w = f64(a["w_pre"]) if a["w_pre"] is not None else np.ones(C)
    out, mag = {}, {}
    dx = dr if dr is not None else np.zeros((rows, C))
    m = np.abs(dx)
    if dn is not None:
        rh = f64(r) * pre[:, None]
        t = dn * w
        dx = dx + pre[:, None] * (t - rh * (t * rh).mean(1, keepdims=True))
        m = m + pre[:, None] * (np.abs(t) + np.abs(rh) * np.abs(t * rh).mean(1, keepdims=True))
        out["dw_pre"], mag["dw_pre"] = (dn * rh).sum(0), np.abs(dn * rh).sum(0)
    out["dx"], mag["dx"] = dx, m
    if y is not None:
        yh = y * post[:, None] if post is not None else y
        wp = f64(a["w_post"]) if a["w_post"] is not None else np.ones(C)
        g = rows_of_gate(f64(a["gate"]), rows) if a["gate"] is not None else np.ones((rows, C))
        s, sm = alpha * g * dx * wp, np.abs(alpha * g * wp) * m
        if post is not None:
            out["dy"] = post[:, None] * (s - yh * (s * yh).mean(1, keepdims=True))
            mag["dy"] = post[:, None] * (sm + np.abs(yh) * (sm * np.abs(yh)).mean(1, keepdims=True))
            out["dw_post"] = (alpha * g * dx * yh).sum(0)
            mag["dw_post"] = (np.abs(alpha * g * yh) * m).sum(0)
        else:
            out["dy"], mag["dy"] = s, sm
        if a["gate"] is not None:
            k = a["gate"].shape[0]
            out["dgate"] = (alpha * dx * yh * wp).reshape(k, rows // k, C).sum(1)
            mag["dgate"] = (np.abs(alpha * yh * wp) * m).reshape(k, rows // k, C).sum(1)
    return out, mag


def check_bwd(amd, a, r, post, pre, alpha, got, x, y, rows):
    ref, mag = ref_bwd(a, r, alpha, f64(post) if post is not None else None, f64(pre))
    dx, dy, dgate, dwp, dwq = got
    check(dx, ref["dx"], K * mag["dx"] + HALF[x] * (1 + K) * np.abs(ref["dx"]), "dx")
    if dy is not None:
        check(dy, ref["dy"], 2 * K * mag["dy"] + HALF[y] * (1 + K) * np.abs(ref["dy"]), "dy")
    for name, t in (("dgate", dgate), ("dw_post", dwp), ("dw_pre", dwq)):
        if t is not None and name in ref:
            check(t, ref[name], (2 * K + (rows + 64) * U) * mag[name], name)


@pytest.mark.parametrize("rows,cols", SHAPES + [(700, 256), (1200, 40)])
@pytest.mark.parametrize("x,y,n", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "f32", "bf16"),
                                   ("bf16", "f32", "bf16")])
def test_backward(amd, rows, cols, x, y, n):
    a = make(rows, cols, x, y, n, seed=rows * 3 + cols)
    r, _, post, pre = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=0.7,
                                     n_dtype=a["n_type"])
    got = amd.block_norm_backward(a["dr"], a["dn"], r, a["y"], a["w_post"], a["w_pre"], post, pre, gate=a["gate"],
                                  alpha=0.7)
    check_bwd(amd, a, r, post, pre, 0.7, got, x, y, rows)


# enough rows for the kernels that stream rows through shared memory
MANY = [(2600, 512), (1300, 1000), (1300, 2048), (700, 2056), (660, 4096), (1301, 1024)]


@pytest.mark.parametrize("rows,cols", MANY)
@pytest.mark.parametrize("x,y,n", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"),
                                   ("bf16", "f32", "f32"), ("bf16", "f32", "bf16")])
@pytest.mark.parametrize("groups", [1, 20])
def test_many_rows(amd, rows, cols, x, y, n, groups):
    rows -= rows % groups
    a = make(rows, cols, x, y, n, groups, seed=rows + 7 * cols)
    r, nn, post, pre = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=0.5, eps=1e-5,
                                      n_dtype=a["n_type"])
    R, N, P, Q, sr, sn = ref_fwd(a, 0.5, 1e-5)
    check(r, R, K * sr + HALF[x] * (1 + K) * np.abs(R), "r")
    check(nn, N, 2 * K * sn + K * np.abs(N) + HALF[n] * (1 + K) * np.abs(N) + K * np.abs(N).max(), "n")
    check(post, P, K * P, "rstd_post")
    check(pre, Q, 2 * K * Q, "rstd_pre")
    got = amd.block_norm_backward(a["dr"], a["dn"], r, a["y"], a["w_post"], a["w_pre"], post, pre, gate=a["gate"],
                                  alpha=0.5)
    check_bwd(amd, a, r, post, pre, 0.5, got, x, y, rows)
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)


# more of them for narrow rows, which stream several at once, and rows that are
# no whole 16 bytes, which stream as the aligned pieces that hold them
STREAMED = [(4900, 512), (2500, 1000), (950, 2056), (4870, 389), (2440, 1013), (2440, 1012), (1300, 2047),
            (640, 3047), (310, 4099), (308, 8191)]


@pytest.mark.parametrize("rows,cols", STREAMED)
@pytest.mark.parametrize("x,y,n", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"),
                                   ("bf16", "f32", "f32")])
@pytest.mark.parametrize("groups", [1, 10])
def test_streamed_rows(amd, rows, cols, x, y, n, groups):
    """As many rows as stream; and each row's results are those of a call of a few."""
    import torch
    rows -= rows % groups
    a = make(rows, cols, x, y, n, groups, seed=rows + 7 * cols)
    if groups == 1:
        a["gate"] = None
    fwd = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=0.5, eps=1e-5,
                         n_dtype=a["n_type"])
    r, nn, post, pre = fwd
    R, N, P, Q, sr, sn = ref_fwd(a, 0.5, 1e-5)
    check(r, R, K * sr + HALF[x] * (1 + K) * np.abs(R), "r")
    check(nn, N, 2 * K * sn + K * np.abs(N) + HALF[n] * (1 + K) * np.abs(N) + K * np.abs(N).max(), "n")
    check(post, P, K * P, "rstd_post")
    check(pre, Q, 2 * K * Q, "rstd_pre")
    got = amd.block_norm_backward(a["dr"], a["dn"], r, a["y"], a["w_post"], a["w_pre"], post, pre, gate=a["gate"],
                                  alpha=0.5)
    check_bwd(amd, a, r, post, pre, 0.5, got, x, y, rows)
    last = slice(rows - 3, rows)
    gate = None if a["gate"] is None else a["gate"][-1:]
    few = amd.block_norm(a["x"][last], a["y"][last], a["w_post"], a["w_pre"], gate=gate, alpha=0.5, eps=1e-5,
                         n_dtype=a["n_type"])
    assert all(torch.equal(p[last], q) for p, q in zip(fwd, few))
    few = amd.block_norm_backward(a["dr"][last], a["dn"][last], r[last], a["y"][last], a["w_post"], a["w_pre"],
                                  post[last], pre[last], gate=gate, alpha=0.5)
    assert torch.equal(got[0][last], few[0]) and torch.equal(got[1][last], few[1])
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)


@pytest.mark.parametrize("cols,pad,off", [(1024, 1, 0), (1024, 0, 3), (1023, 2, 5), (1016, 16, 8)])
def test_streamed_strides_and_alignment(amd, cols, pad, off):
    """Rows with a stride and bases off 16 bytes, in place: the dense result, to the bit
    where both deal the channels to threads alike, and nothing outside the rows is
    written."""
    import torch
    rows, ld = 2500, cols + pad
    a = make(rows, cols, "bf16", "f32", "bf16", 2, seed=6)

    def spread(t):
        buf = torch.full((rows * ld + off + 8,), 5.0, dtype=t.dtype, device="cuda")
        v = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
        v.copy_(t)
        return buf, v

    def untouched(buf, v):
        v.fill_(5.0)
        return bool((buf == 5.0).all())
    r, n, post, pre = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], n_dtype=a["n_type"])
    back = amd.block_norm_backward(a["dr"], a["dn"], r, a["y"], a["w_post"], a["w_pre"], post, pre, gate=a["gate"])
    (xb, x), (yb, y), (nb, nv) = spread(a["x"]), spread(a["y"]), spread(n * 0)
    d = amd.BlockNormDesc(rows=rows, cols=cols, gate_rows=rows // 2, alpha=1.0, eps=1e-6, x_type=1, y_type=0, n_type=1,
                          ldx=ld, ldy=ld, ldr=ld, ldn=ld, lddr=ld, lddn=ld, lddx=ld, lddy=ld)
    amd.amsim_block_norm_fwd(d, x, y, a["gate"], a["w_post"], a["w_pre"], x, nv, None, None)
    same = (lambda p, q: torch.allclose(p.float(), q.float(), rtol=2.0 ** -7, atol=2.0 ** -7)) if cols % 4 == 0 and (
        ld % 4 or off % 4) else torch.equal
    assert same(x, r) and same(nv, n)
    assert untouched(xb, x) and untouched(yb, y) and untouched(nb, nv)
    (rb, rv), (yb, y), (drb, dr), (dnb, dn) = (spread(t) for t in (r, a["y"], a["dr"], a["dn"]))
    ws = amd.workspace(amd.amsim_block_norm_workspace_size(d))
    sums = [torch.empty_like(a["gate"]), torch.empty_like(a["w_post"]), torch.empty_like(a["w_pre"])]
    amd.amsim_block_norm_bwd(d, dr, dn, rv, y, a["gate"], a["w_post"], a["w_pre"], post, pre, dr, y, *sums, ws=ws)
    check_bwd(amd, a, r, post, pre, 1.0, [dr, y, *sums], "bf16", "f32", rows)
    assert same(dr, back[0]) and same(y, back[1])
    assert untouched(drb, dr) and untouched(yb, y)


@pytest.mark.parametrize("drop", ["dr", "dn", "y", "w_post", "w_pre", "gate"])
def test_many_rows_without_parts(amd, drop):
    a = make(2600, 512, "f32", "bf16", "f32", 4, seed=9)
    a[drop] = None
    if drop == "y":
        a["w_post"] = a["gate"] = None
    r, n, post, pre = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=0.7,
                                     n_dtype=a["n_type"])
    R, N, P, Q, sr, sn = ref_fwd(a, 0.7, 1e-6)
    check(r, R, K * sr, "r")
    check(n, N, 4 * K * sn + K * np.abs(N).max(), "n")
    got = amd.block_norm_backward(a["dr"], a["dn"], r, a["y"], a["w_post"], a["w_pre"], post, pre, gate=a["gate"],
                                  alpha=0.7)
    check_bwd(amd, a, r, post, pre, 0.7, got, "f32", "bf16", 2600)


@pytest.mark.parametrize("groups", [2, 5, 300, 600])
def test_backward_shared_gates(amd, groups):
    """A gate row's gradient is the sum over the rows that share it, few or one."""
    a = make(600, 96, "f32", "f32", "f32", groups, seed=groups)
    r, _, post, pre = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=0.3)
    got = amd.block_norm_backward(a["dr"], a["dn"], r, a["y"], a["w_post"], a["w_pre"], post, pre, gate=a["gate"],
                                  alpha=0.3)
    check_bwd(amd, a, r, post, pre, 0.3, got, "f32", "f32", 600)


@pytest.mark.parametrize("drop", ["dr", "dn", "y", "w_post", "w_pre", "gate"])
def test_backward_without_parts(amd, drop):
    a = make(40, 120, "f32", "bf16", "f32", 4, seed=9)
    a[drop] = None
    if drop == "y":
        a["w_post"] = a["gate"] = None
    r, _, post, pre = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=0.7,
                                     n_dtype=a["n_type"])
    got = amd.block_norm_backward(a["dr"], a["dn"], r, a["y"], a["w_post"], a["w_pre"], post, pre, gate=a["gate"],
                                  alpha=0.7)
    check_bwd(amd, a, r, post, pre, 0.7, got, "f32", "bf16", 40)
    if drop == "dn":
        assert not got[4].any()


def test_backward_any_scratch(amd):
    """Fewer row shares with less scratch, one with none; each deterministic,
    and all within the bounds."""
    import torch
    a = make(900, 200, "f32", "f32", "f32", 3, seed=2)
    r, _, post, pre = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=0.7)
    d = amd.BlockNormDesc(rows=900, cols=200, gate_rows=300, alpha=0.7)
    full = amd.amsim_block_norm_workspace_size(d)
    assert full > 4 * 200 * 4
    for nbytes in (full, full // 3, 5 * 800, 800, 0):
        outs = []
        for _ in range(2):
            o = [torch.full_like(r, 7.0), torch.full_like(r, 7.0), torch.full((3, 200), 7.0, device="cuda"),
                 torch.full((200,), 7.0, device="cuda"), torch.full((200,), 7.0, device="cuda")]
            ws = torch.full((max(nbytes, 4),), 255, dtype=torch.uint8, device="cuda")
            amd.amsim_block_norm_bwd(d, a["dr"], a["dn"], r, a["y"], a["gate"], a["w_post"], a["w_pre"], post, pre,
                                     *o, ws=ws if nbytes else None, ws_bytes=nbytes)
            outs.append(o)
        check_bwd(amd, a, r, post, pre, 0.7, outs[0], "f32", "f32", 900)
        assert all(torch.equal(p, q) for p, q in zip(*outs))


@pytest.mark.parametrize("cols,pad,off", [(64, 8, 0), (64, 3, 0), (50, 6, 2), (128, 0, 1)])
def test_strides_and_alignment(amd, cols, pad, off):
    """Rows with a stride, and bases off 16 bytes, give the dense result, and
    nothing outside the rows is written."""
    import torch
    a = make(9, cols, "bf16", "f32", "bf16", 3, seed=6)

    def spread(t):
        buf = torch.full((9 * (cols + pad) + off + 8,), 5.0, dtype=t.dtype, device="cuda")
        v = buf[off:off + 9 * (cols + pad)].view(9, cols + pad)[:, :cols]
        v.copy_(t)
        return buf, v
    x, y, dr, dn = (spread(a[k])[1] for k in ("x", "y", "dr", "dn"))
    dense = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], n_dtype=a["n_type"])
    got = amd.block_norm(x, y, a["w_post"], a["w_pre"], gate=a["gate"], n_dtype=a["n_type"])
    R, N, P, Q, sr, sn = ref_fwd(a, 1.0, 1e-6)
    check(got[0], R, K * sr + HALF["bf16"] * (1 + K) * np.abs(R), "r")
    # strided outputs through the C ABI
    rb, rv = spread(torch.zeros_like(a["x"]))
    nb, nv = spread(torch.zeros_like(a["x"]))
    d = amd.BlockNormDesc(rows=9, cols=cols, gate_rows=3, alpha=1.0, eps=1e-6, x_type=1, y_type=0, n_type=1,
                          ldx=x.stride(0), ldy=y.stride(0), ldr=rv.stride(0), ldn=nv.stride(0))
    amd.amsim_block_norm_fwd(d, x, y, a["gate"], a["w_post"], a["w_pre"], rv, nv, None, None)
    assert torch.equal(rv, got[0]) and torch.equal(nv, got[1])
    for buf, v in ((rb, rv), (nb, nv)):
        v.fill_(5.0)
        assert bool((buf == 5.0).all())
    back = amd.block_norm_backward(dr, dn, dense[0], y, a["w_post"], a["w_pre"], dense[2], dense[3], gate=a["gate"])
    check_bwd(amd, a, dense[0], dense[2], dense[3], 1.0, back, "bf16", "f32", 9)


def test_in_place(amd):
    """r over x, n over y; dx over dr, dy over y."""
    import torch
    a = make(50, 256, "f32", "f32", "f32", 2, seed=1)
    want = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"])
    x, y = a["x"].clone(), a["y"].clone()
    d = amd.BlockNormDesc(rows=50, cols=256, gate_rows=25, alpha=1.0, eps=1e-6)
    amd.amsim_block_norm_fwd(d, x, y, a["gate"], a["w_post"], a["w_pre"], x, y, None, None)
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])
    back = amd.block_norm_backward(a["dr"], a["dn"], want[0], a["y"], a["w_post"], a["w_pre"], want[2], want[3],
                                   gate=a["gate"])
    dr, y = a["dr"].clone(), a["y"].clone()
    ws = amd.workspace(amd.amsim_block_norm_workspace_size(d))
    amd.amsim_block_norm_bwd(d, dr, a["dn"], want[0], y, a["gate"], a["w_post"], a["w_pre"], want[2], want[3], dr, y,
                             None, None, None, ws=ws)
    assert torch.equal(dr, back[0]) and torch.equal(y, back[1])


def test_special_values_stay_in_their_row(amd):
    """A zero row has a finite norm through eps (and a zero one through eps 0
    is its own affair); NaN and infinity spoil their row alone."""
    import torch
    a = make(8, 64, seed=3)
    clean = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"])
    for k in ("x", "y"):
        a[k][2] = 0.0
    a["x"][5, 3] = float("nan")
    a["y"][6, 0] = float("inf")
    r, n, p, q = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"])
    assert not r[2].any() and not n[2].any() and bool(torch.isfinite(torch.stack([p[2], q[2]])).all())
    assert bool(torch.isnan(n[5]).all()) and not bool(torch.isfinite(r[6, 0]))
    keep = [0, 1, 3, 4, 7]
    assert torch.equal(r[keep], clean[0][keep]) and torch.equal(n[keep], clean[1][keep])


def test_no_rows(amd):
    import torch
    a = make(0, 24)
    d = amd.BlockNormDesc(rows=0, cols=24, alpha=1.0)
    dw = torch.full((24,), 3.0, device="cuda")
    amd.amsim_block_norm_bwd(d, a["dr"], a["dn"], a["x"], a["y"], None, a["w_post"], a["w_pre"], None, None, a["x"],
                             a["y"], None, dw, None)
    assert not dw.any()


def test_gradient_against_differences(amd):
    """<gradient, direction> against central differences of the formula in 64
    bits: L = sum(r cr) + sum(n cn).  The differences' own error is O(h^2), the
    gradient's K of the magnitudes."""
    a = make(10, 48, groups=2, seed=12)
    alpha, eps = 0.7, 1e-3
    r, n, post, pre = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"], alpha=alpha, eps=eps)
    got = amd.block_norm_backward(a["dr"], a["dn"], r, a["y"], a["w_post"], a["w_pre"], post, pre, gate=a["gate"],
                                  alpha=alpha)
    base = {k: f64(a[k]) for k in ("x", "y", "gate", "w_post", "w_pre")}
    dr, dn = f64(a["dr"]), f64(a["dn"])

    def loss(v):
        yh = v["y"] / np.sqrt((v["y"] ** 2).mean(1, keepdims=True) + eps)
        rr = v["x"] + alpha * rows_of_gate(v["gate"], 10) * yh * v["w_post"]
        return (rr * dr).sum() + (rr / np.sqrt((rr ** 2).mean(1, keepdims=True) + eps) * v["w_pre"] * dn).sum()
    rng = np.random.default_rng(0)
    for name, grad in zip(("x", "y", "gate", "w_post", "w_pre"), got):
        d = rng.standard_normal(base[name].shape)
        h = 1e-5
        up, dn_ = dict(base), dict(base)
        up[name], dn_[name] = base[name] + h * d, base[name] - h * d
        want = (loss(up) - loss(dn_)) / (2 * h)
        have = (f64(grad) * d).sum()
        assert abs(have - want) <= 200 * K * np.abs(f64(grad) * d).sum() + 1e-6 * abs(want), name


def test_other_stream(amd):
    import torch
    a = make(64, 512, "bf16", "bf16", "bf16", 4, seed=8)
    want = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = amd.block_norm(a["x"], a["y"], a["w_post"], a["w_pre"], gate=a["gate"])
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in itertools.islice(zip(got, want), 4))


def test_offsets_past_32_bits(amd):
    """2^31 and more elements: the last rows are the ones a small call computes."""
    import torch
    rows, cols = 530_000, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((16, cols), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    x[-16:] = tail.to(torch.bfloat16)
    w = torch.ones(cols, device="cuda")
    r, n, post, pre = amd.block_norm(x, x, w, w)
    small = amd.block_norm(x[-16:], x[-16:], w, w)
    assert torch.equal(r[-16:], small[0]) and torch.equal(n[-16:], small[1]) and torch.equal(pre[-16:], small[3])
    dx, dy, _, dwp, dwq = amd.block_norm_backward(x, x, r, x, w, w, post, pre)
    sb = amd.block_norm_backward(x[-16:], x[-16:], r[-16:], x[-16:], w, w, post[-16:], pre[-16:])
    assert torch.equal(dx[-16:], sb[0]) and torch.equal(dy[-16:], sb[1])
    assert torch.allclose(dwq, sb[4], rtol=1e-5, atol=1e-5)
