"""The vocabulary loss against its formulas in 64 bits.

Bounds.  A logit is a sum of exact products; every 16 products the tensor cores
add with truncation, so its error is at most ez = (D / 16 + 4) 2^-23 times the
sum of the products' magnitudes.  lse adds the exponentials' error (2^-20 with
the sums') and its rounding: el = max ez + 2^-20 + 4 u |lse|.  A probability
carries its logit's and lse's error and its 16-bit code's (2^-12 of it); G is
rounded to bf16 (2^-8 of it); dh and dw add the truncated sums (n / 16 + 4)
2^-23 of their magnitudes and their own rounding (2^-8 of the result)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IGNORE = -100


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, V, D, seed=0, ignored=0.2, scale=2.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    h = torch.randn((T, D), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((V, D), generator=g) * (scale / D ** 0.5)).to(torch.bfloat16).cuda()
    t = torch.randint(0, V, (T,), generator=g)
    t[torch.rand(T, generator=g) < ignored] = IGNORE
    return h, w, t.cuda()


def reference(h, w, t, weight=None, mean=True):
    """Values and bounds of loss, row losses, lse, dh, dw."""
    H, W, t = f64(h), f64(w), t.cpu().numpy()
    T, D = H.shape
    V = W.shape[0]
    counts = t != IGNORE
    valid = counts & (t >= 0) & (t < V)
    a = np.where(counts, 1.0 if weight is None else f64(weight), 0.0)
    z = H @ W.T
    ez = (D / 16 + 4) * 2.0 ** -23 * (np.abs(H) @ np.abs(W).T)
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    el = ez.max(1) + 2.0 ** -20 + 4 * U * np.abs(lse)
    at = np.where(valid, t, 0)
    rows = np.arange(T)
    row = np.where(valid, lse - z[rows, at], np.where(counts, np.nan, 0.0))
    er = el + ez[rows, at] + 4 * U * (np.abs(lse) + np.abs(z[rows, at]))
    A = a.sum() if mean else 1.0
    s = 1.0 / A if A else 0.0
    loss = (np.where(counts, row, 0.0) * a).sum() * s
    eloss = (np.where(counts, er, 0.0) * np.abs(a)).sum() * s + 4 * U * abs(loss)
    p = np.exp(z - lse[:, None])
    g = p.copy()
    g[rows[valid], t[valid]] -= 1.0
    b = np.where(valid, a, 0.0)[:, None]
    eg = np.abs(b) * (p * (2.0 ** -12 * 1.01 + ez + el[:, None] + 2.0 ** -20) + 2.0 ** -8 * np.abs(g) + 2e-14)
    g = g * b

    def product(x, ex, y, n):
        out = s * (x @ y)
        mag = (np.abs(x) + ex) @ np.abs(y)
        return out, s * (ex @ np.abs(y) + (n / 16 + 4) * 2.0 ** -23 * mag) * (1 + 2.0 ** -8) + \
            2.0 ** -8 * np.abs(out) + 1e-38
    dh, edh = product(g, eg, W, V)
    dw, edw = product(g.T, eg.T, H, T)
    return [(np.array([loss]), np.array([eloss])), (row, np.where(valid, er, 0.0)), (lse, el), (dh, edh), (dw, edw)]


def compare(got, ref, what=""):
    for name, x, (want, tol) in zip(("loss", "row_loss", "lse", "dh", "dw"), got, ref):
        x = f64(x)
        nan = np.isnan(want)
        assert np.array_equal(nan, np.isnan(x)), f"{what} {name}: NaN pattern"
        err = np.abs(x - want)[~nan]
        assert np.all(err <= np.broadcast_to(tol, want.shape)[~nan]), \
            f"{what} {name}: error {err.max():.3e}, over its bound by {(err - np.broadcast_to(tol, want.shape)[~nan]).max():.3e}"


SHAPES = [(1, 1, 1), (1, 2, 8), (1, 1000, 64), (2, 129, 24), (3, 128, 100), (7, 257, 72), (24, 8192, 256),
          (127, 1001, 130), (128, 512, 64), (129, 640, 1032), (200, 3000, 2056), (300, 127, 8), (513, 2000, 200),
          (1000, 300, 96), (33, 20000, 40), (64, 4099, 4096)]


@pytest.mark.parametrize("T,V,D", SHAPES)
def test_loss_and_gradients(amd, T, V, D):
    h, w, t = make(T, V, D, seed=T + V)
    ref = reference(h, w, t)
    compare(amd.vocab_loss_grad(h, w, t), ref, "grad")
    compare(amd.vocab_loss(h, w, t), ref, "loss")
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)


@pytest.mark.parametrize("mean", [True, False])
def test_row_weights(amd, mean):
    import torch
    h, w, t = make(150, 900, 80, seed=3)
    a = torch.rand(150, generator=torch.Generator().manual_seed(1)).cuda() * 2
    a[5] = 0.0
    a[6] = -0.5
    got = amd.vocab_loss_grad(h, w, t, row_weight=a, reduction="mean" if mean else "sum")
    compare(got, reference(h, w, t, a, mean))


def test_masked_and_invalid_targets(amd):
    """No token that counts: loss and gradients are zero.  A target outside the
    vocabulary: NaN row loss and loss, no gradient, the other rows as they are."""
    import torch
    h, w, t = make(40, 300, 64, seed=4, ignored=0.0)
    none = torch.full_like(t, IGNORE)
    loss, row, lse, dh, dw = amd.vocab_loss_grad(h, w, none)
    assert not loss.any() and not row.any() and not dh.any() and not dw.any() and bool(torch.isfinite(lse).all())
    t[3], t[17] = 300, -7
    got = amd.vocab_loss_grad(h, w, t)
    ref = reference(h, w, t)
    ref[0] = (np.array([np.nan]), np.array([0.0]))
    compare(got, ref)
    assert not got[3][3].any() and not got[3][17].any()
    other = amd.vocab_loss(h, w, torch.where(t < 0, 5, t.clamp(max=299)), ignore_index=5)
    assert not other[1][17].any()                         # a token id as ignore_index


def test_scratch_chunks(amd):
    """Less scratch takes the tokens in more chunks: the same losses to the
    bit per row, gradients within the bounds, every run the same bits; less
    than the least is refused."""
    import torch
    T, V, D = 700, 1500, 136
    h, w, t = make(T, V, D, seed=6)
    d = amd.VocabLossDesc(tokens=T, vocab=V, dim=D, ignore_index=IGNORE, reduction=0)
    ref = reference(h, w, t)
    full, least = amd.amsim_vocab_loss_workspace_size(d, 1), amd.amsim_vocab_loss_workspace_min(d, 1)
    rows = None
    for nbytes in (full, (full + least) // 2, least):
        runs = []
        for _ in range(2):
            out = [torch.full((n,), 3.0, device="cuda") for n in (1, T, T)]
            out += [torch.full((n, D), 3.0, dtype=torch.bfloat16, device="cuda") for n in (T, V)]
            ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
            amd.amsim_vocab_loss_grad(d, h, w, t, None, *out, ws=ws)
            runs.append(out)
        compare(runs[0], ref, f"{nbytes} bytes")
        assert all(torch.equal(a, b) for a, b in zip(*runs))
        if rows is not None:
            assert torch.equal(rows, runs[0][1])
        rows = runs[0][1]
    with pytest.raises(amd.AmsimError) as e:
        amd.amsim_vocab_loss_grad(d, h, w, t, None, *runs[0], ws=ws, ws_bytes=least // 2)
    assert e.value.status == amd.AMSIM_EINVAL
    d0 = amd.amsim_vocab_loss_workspace_min(d, 0)
    out = [torch.empty(n, device="cuda") for n in (1, T, T)]
    amd.amsim_vocab_loss(d, h, w, t, None, *out, ws=amd.workspace(d0))
    compare(out, ref)


@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (0, 1), (5, 2)])
def test_strides_and_alignment(amd, pad, off):
    """Rows with strides and bases that copies cannot take directly; strided
    gradients leave what lies between their rows alone."""
    import torch
    T, V, D = 70, 400, 48
    h, w, t = make(T, V, D, seed=7)

    def spread(x):
        n = x.shape[0]
        buf = torch.full((n * (D + pad) + off + 8,), 5.0, dtype=x.dtype, device="cuda")
        v = buf[off:off + n * (D + pad)].view(n, D + pad)[:, :D]
        v.copy_(x)
        return buf, v
    hs, ws_ = spread(h)[1], spread(w)[1]
    ref = reference(h, w, t)
    compare(amd.vocab_loss_grad(hs, ws_, t), ref, "strided")
    compare(amd.vocab_loss(hs, ws_, t), ref, "strided")
    (hb, dh), (wb, dw) = spread(torch.zeros_like(h)), spread(torch.zeros_like(w))
    d = amd.VocabLossDesc(tokens=T, vocab=V, dim=D, ignore_index=IGNORE, reduction=0, ld_h=hs.stride(0),
                          ld_w=ws_.stride(0), ld_dh=dh.stride(0), ld_dw=dw.stride(0))
    out = [torch.empty(n, device="cuda") for n in (1, T, T)]
    amd.amsim_vocab_loss_grad(d, hs, ws_, t, None, *out, dh, dw, ws=amd.workspace(amd.amsim_vocab_loss_workspace_size(d, 1)))
    compare(out + [dh, dw], ref, "strided outputs")
    for buf, v in ((hb, dh), (wb, dw)):
        v.fill_(5.0)
        assert bool((buf == 5.0).all())


def test_special_values(amd):
    """Large logits (far past exp's range) keep finite results; a non-finite
    hidden state spoils its own row's loss and gradient only."""
    import torch
    h, w, t = make(60, 500, 64, seed=8, scale=60.0, ignored=0.0)
    compare(amd.vocab_loss_grad(h, w, t), reference(h, w, t), "large logits")
    h, w, t = make(60, 500, 64, seed=9, ignored=0.0)
    clean = amd.vocab_loss_grad(h, w, t)
    h[7, 5] = float("nan")
    h[9, 1] = float("inf")
    loss, row, lse, dh, dw = amd.vocab_loss_grad(h, w, t)
    keep = [i for i in range(60) if i not in (7, 9)]
    assert torch.equal(row[keep], clean[1][keep]) and torch.equal(lse[keep], clean[2][keep])
    assert torch.equal(dh[keep], clean[3][keep])
    assert bool(torch.isnan(torch.stack([loss[0], row[7], row[9], lse[7]])).all())
    t[7] = t[9] = IGNORE                                  # masked out, they spoil nothing but their lse
    loss, row, lse, dh, dw = amd.vocab_loss_grad(h, w, t)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(row).all()) and bool(torch.isfinite(dh).all())


def test_gradient_against_differences(amd):
    """<gradient, direction> against central differences of the formula in 64
    bits; the gradient's own bound covers the difference (h^2 terms are below it)."""
    h, w, t = make(20, 90, 32, seed=10)
    ref = reference(h, w, t)
    _, _, _, dh, dw = amd.vocab_loss_grad(h, w, t)
    H, W, tt = f64(h), f64(w), t.cpu().numpy()
    keep = tt != IGNORE

    def loss(H, W):
        z = H @ W.T
        top = z.max(1)
        return (top + np.log(np.exp(z - top[:, None]).sum(1)) - z[np.arange(20), np.where(keep, tt, 0)])[keep].mean()
    rng = np.random.default_rng(1)
    for which, grad, tol in ((0, dh, ref[3][1]), (1, dw, ref[4][1])):
        d = rng.standard_normal((H, W)[which].shape)
        e = 1e-5
        plus = loss(H + e * d, W) if which == 0 else loss(H, W + e * d)
        minus = loss(H - e * d, W) if which == 0 else loss(H, W - e * d)
        want, have = (plus - minus) / (2 * e), (f64(grad) * d).sum()
        assert abs(have - want) <= (tol * np.abs(d)).sum() + 1e-7


def test_no_tokens(amd):
    import torch
    h = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((10, 16), dtype=torch.bfloat16, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, row, lse, dh, dw = amd.vocab_loss_grad(h, w, t)
    assert float(loss) == 0.0 and row.numel() == 0 and not dw.any()
    assert float(amd.vocab_loss(h, w, t)[0]) == 0.0


def test_other_stream_and_graph(amd):
    """On a side stream, and replayed from a captured graph over new inputs."""
    import torch
    h, w, t = make(130, 700, 64, seed=11)
    want = amd.vocab_loss_grad(h, w, t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = amd.vocab_loss_grad(h, w, t)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    hs = torch.zeros_like(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = amd.vocab_loss_grad(hs, w, t)
    for _ in range(2):
        hs.copy_(h)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        hs.zero_()


def test_offsets_past_32_bits(amd):
    """More than 2^31 exponentials in scratch, and several chunks: rows at the
    ends against 64 bits."""
    import torch
    T, V, D = 17_000, 131_072, 64
    h, w, t = make(T, V, D, seed=12)
    loss, row, lse, dh, dw = amd.vocab_loss_grad(h, w, t)
    pick = np.r_[0:3, 8191:8194, 16383:16386, T - 3:T]
    ref = reference(h[pick], w, t[pick])
    compare((loss, row[pick], lse[pick]), [(f64(loss), np.array([0.0]))] + ref[1:3], "rows")
    counts = int((t != IGNORE).sum())
    mine = int((t[pick] != IGNORE).sum())
    dh_ref, dh_tol = ref[3]
    err = np.abs(f64(dh[pick]) * counts - dh_ref * mine)
    assert np.all(err <= dh_tol * mine + 2.0 ** -8 * np.abs(dh_ref * mine))
    z = h.double() @ w[-2:].double().t()                  # the last rows of dw, from the rows' own lse
    g = torch.exp(z - lse.double()[:, None]) * (t != IGNORE)[:, None]
    for j in range(2):
        g[t == V - 2 + j, j] -= 1.0
    want = f64((g.t() @ h.double()) / counts)
    mag = f64((g.abs().t() @ h.double().abs()) / counts)
    assert np.all(np.abs(f64(dw[-2:]) - want) <= mag * (2.0 ** -8 + 2.0 ** -11 + T / 16 * 2.0 ** -23) +
                  2.0 ** -8 * np.abs(want))
