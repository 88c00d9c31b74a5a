"""The attention softmax and its gradient against the definition in 64 bits.

u = 2^-24.  A logit a = s + bias is off by u |a|, its difference to the row's
maximum by u (|a| + |max| + |a - max|) in all, so with A the row's largest |a|
an exponential is within 4 A u + 4 u (the function itself), relative; the sum
of a row takes at most keys / 1024 + 64 additions one after the other in a
thread and its tree, and three more products and quotients follow: a
probability is within E = (4 A + 80 + keys / 1024) u of its value.  The
gradient's sum over a row is within (E + (64 + keys / 1024) u) of the sum of
its terms' magnitudes; dtable adds one u for each of its rows at most."""
import numpy as np
import pytest

from philox_reference import stays

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def reference(scores, table, buckets, lengths, causal, offset, p, seed, call, dprobs=None):
    """probs, stats, logits, and with dprobs (dscores, dtable) and their bounds."""
    s = scores.double().cpu().numpy()
    B, H, Q, K = s.shape
    off = np.broadcast_to(offset.cpu().numpy() if hasattr(offset, "cpu") else offset, (B,)).astype(np.int64)
    pos = off[:, None] + np.arange(Q)
    dist = np.arange(K) - pos[..., None]                                  # [B, Q, K]
    a = s
    which = None
    if buckets is not None:
        D = buckets.numel() // 2
        which = buckets.cpu().numpy()[np.clip(dist, -D, D) + D]
    if table is not None:
        t = table.double().cpu().numpy()
        ok = (which >= 0) & (which < t.shape[0])
        a = s + np.where(ok[..., None], t[np.where(ok, which, 0)], 0.0).transpose(0, 3, 1, 2)
    see = np.ones((B, 1, Q, K), bool)
    if lengths is not None:
        see = see & (np.arange(K) < lengths.cpu().numpy()[:, None, None, None])
    if causal:
        see = see & (dist <= 0)[:, None]
    see = np.broadcast_to(see, s.shape)
    a = np.where(see, a, -np.inf)
    top = a.max(-1, keepdims=True, initial=-np.inf)
    e = np.exp(a - np.where(np.isneginf(top), 0.0, top))
    total = e.sum(-1, keepdims=True)
    inv = np.where(total == 0, 0.0, 1.0 / np.where(total == 0, 1.0, total))
    P = np.where(see, e * inv, 0.0)
    big = np.where(np.isfinite(a), np.abs(a), 0.0).max(-1, keepdims=True, initial=0.0)
    E = (4 * big + 80 + K / 1024) * U
    keep = stays(B * H * Q, K, p, call, seed).reshape(s.shape) if p else np.ones(s.shape, bool)
    out = dict(probs=np.where(keep, P / (1 - p), 0.0), stats=np.concatenate([top, inv], -1), E=E, P=P)
    if dprobs is not None:
        g = np.where(see & keep, dprobs.double().cpu().numpy(), 0.0) / (1 - p)
        terms = np.abs(P * g).sum(-1, keepdims=True)
        dot = (P * g).sum(-1, keepdims=True)
        ds = P * (g - dot)
        tol = P * ((2 * E + (64 + K / 1024) * U) * (terms + np.abs(g)) + 4 * U * (np.abs(g) + np.abs(dot)))
        out.update(ds=ds, ds_tol=tol)
        if buckets is not None and table is not None:
            dt, dt_tol = np.zeros(table.shape), np.zeros(table.shape)
            w = np.broadcast_to(which[:, None], s.shape)
            for k in range(table.shape[0]):
                m = w == k
                dt[k] = np.where(m, ds, 0).sum((0, 2, 3))
                dt_tol[k] = np.where(m, tol + (B * Q + 64 + K / 32) * U * np.abs(ds), 0).sum((0, 2, 3))
            out.update(dt=dt, dt_tol=dt_tol)
    return out


def near(got, ref, tol, what):
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol + 2.0 ** -120), f"{what}: error {np.nanmax(err):.3e}, over its bound by " \
                                             f"{np.nanmax(err - tol):.3e}"


def make(B, H, Q, K, seed=0, bias=None, buckets=32, distance=128):
    import torch
    import approximate_multiplier_dnn_gb300 as am
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = torch.randn((B, H, Q, K), generator=g, device="cuda") * 2
    d = torch.randn((B, H, Q, K), generator=g, device="cuda")
    t = b = None
    if bias:
        t = torch.randn((buckets, H), generator=g, device="cuda")
        b = am.relative_buckets(buckets, distance, bias == "both").cuda()
    return s, d, t, b


def both_ways(amd, s, d, t, b, p=0.0, seed=77, call=5, table_grad=True, **kw):
    """Forward and backward against the reference, the gradient from probs and from scores."""
    import torch
    ref = reference(s, t, b, kw.get("lengths"), kw.get("causal", False), kw.get("offset", 0), p, seed, call, d)
    args = dict(table=t, buckets=b, p=p, seed=seed, call=call, **kw)
    probs, stats = amd.attention_softmax(s, **args)
    near(probs, ref["probs"], ref["probs"] * ref["E"], "probs")
    gone = ref["probs"] == 0
    assert not probs.cpu().numpy()[gone & (ref["P"] == 0)].any() and not probs.cpu().numpy()[gone & (ref["P"] > 0)].any()
    top, inv = stats[..., 0].double().cpu().numpy(), stats[..., 1].double().cpu().numpy()
    live = np.isfinite(ref["stats"][..., 0])
    assert np.array_equal(np.isneginf(top), ~live) and not inv[~live].any()
    assert np.all(np.abs(top - ref["stats"][..., 0])[live] <= U * np.abs(ref["stats"][..., 0][live]))
    assert np.all(np.abs(inv - ref["stats"][..., 1]) <= ref["E"][..., 0] * ref["stats"][..., 1])
    ways = [dict(scores=s, stats=stats)] + ([dict(probs=probs)] if not p else [])
    for way in ways:
        ds, dt = amd.attention_softmax_backward(d, table_grad=table_grad, **way, **args)
        near(ds, ref["ds"], ref["ds_tol"], "dscores")
        assert not ds.cpu().numpy()[ref["P"] == 0].any()
        if t is None or not table_grad:
            assert dt is None
        else:
            near(dt, ref["dt"], ref["dt_tol"], "dtable")
        again = amd.attention_softmax_backward(d, table_grad=table_grad, **way, **args)
        assert torch.equal(again[0], ds) and (dt is None or torch.equal(again[1], dt))
    return probs, stats


# a warp, a block and a loop over each row; odd and even
KEYS = [1, 2, 3, 5, 31, 64, 127, 128, 129, 255, 512, 777, 1000, 1024, 1025, 1028, 2050, 4096, 4099]


@pytest.mark.parametrize("keys", KEYS)
@pytest.mark.parametrize("bias", [None, "both"])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_rows(amd, keys, bias, p):
    both_ways(amd, *make(2, 3, 13, keys, keys, bias), p=p)


@pytest.mark.parametrize("keys", [16384, 16387, 20000, 32768, 40001, 131072, 200001, 262144, 300000])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_long_rows(amd, keys, p):
    both_ways(amd, *make(1, 2, 3, keys, keys, "past"), p=p, offset=keys - 3, causal=True)


@pytest.mark.parametrize("queries,keys,offset", [(70, 70, 0), (33, 200, 167), (300, 300, 0), (5, 9, -3), (9, 2000, 1500)])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_causal(amd, queries, keys, offset, p):
    """Rows before the first key (a negative offset) see nothing and are zeros."""
    probs, _ = both_ways(amd, *make(2, 4, queries, keys, 1, "past"), causal=True, offset=offset, p=p)
    if offset < 0:
        assert not probs[:, :, :-offset].any()


@pytest.mark.parametrize("keys", [1, 6, 100, 999, 1531, 5000])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(amd, keys, causal):
    """Lengths of zero, below zero and beyond the keys; what is not seen may be anything."""
    import torch
    s, d, t, b = make(6, 2, 7, keys, 2, "both")
    n = torch.tensor([keys, 0, -3, keys + 5, (keys + 1) // 2, 1], dtype=torch.int32, device="cuda")
    hidden = torch.arange(keys, device="cuda") >= n.view(-1, 1, 1, 1)
    clean, _ = both_ways(amd, s.masked_fill(hidden, 0), d.masked_fill(hidden, 0), t, b, lengths=n, causal=causal)
    for bad in (float("nan"), float("inf"), torch.finfo(torch.float32).min):
        s2, d2 = s.masked_fill(hidden, bad), d.masked_fill(hidden, bad)
        kw = dict(table=t, buckets=b, lengths=n, causal=causal)
        probs, stats = amd.attention_softmax(s2, **kw)
        assert torch.equal(probs, clean)
        ds, dt = amd.attention_softmax_backward(d2, scores=s2, stats=stats, **kw)
        assert bool(torch.isfinite(ds).all()) and bool(torch.isfinite(dt).all())


@pytest.mark.parametrize("keys", [40, 1300, 40000])
def test_values_at_the_type_s_ends(amd, keys):
    """-infinity among the scores has no weight, a row of it is zeros; a row of
    the lowest value is uniform; a NaN or +infinity makes its own row NaN."""
    import torch
    s, d, _, _ = make(1, 1, 7, keys, 3)
    low = torch.finfo(torch.float32).min
    s[0, 0, 0, ::2] = -float("inf")
    s[0, 0, 1] = -float("inf")
    s[0, 0, 2] = low
    s[0, 0, 3, 5] = float("nan")
    s[0, 0, 4, 7] = float("inf")
    s[0, 0, 5] = low
    s[0, 0, 5, 3] = 1.0
    probs, stats = amd.attention_softmax(s)
    assert not probs[0, 0, 0, ::2].any() and abs(float(probs[0, 0, 0].double().sum()) - 1) < 1e-5
    assert not probs[0, 0, 1].any()
    assert np.allclose(probs[0, 0, 2].cpu().numpy(), 1 / keys, rtol=1e-5)
    assert bool(torch.isnan(probs[0, 0, 3]).all()) and bool(torch.isnan(probs[0, 0, 4]).all())
    assert float(probs[0, 0, 5, 3]) == 1.0 and float(probs[0, 0, 5].sum()) == 1.0
    assert bool(torch.isfinite(probs[0, 0, 6]).all())
    ds, _ = amd.attention_softmax_backward(d, scores=s, stats=stats)
    assert not ds[0, 0, 1].any() and bool(torch.isnan(ds[0, 0, 3]).all())
    assert bool(torch.isfinite(ds[0, 0, [0, 1, 2, 5, 6]]).all())


@pytest.mark.parametrize("batch,heads,keys", [(1, 1, 1), (3, 5, 100), (2, 16, 4096), (4, 3, 33333)])
def test_single_token(amd, batch, heads, keys):
    """One query per sequence at its own place of the cache: as that row of the whole sequence."""
    import torch
    s, d, t, b = make(batch, heads, 1, keys, 4, "past")
    g = torch.Generator().manual_seed(1)
    n = torch.randint(1, keys + 1, (batch,), generator=g).to(torch.int32).cuda()
    both_ways(amd, s, d, t, b, lengths=n, offset=n - 1, causal=True)
    probs, _ = amd.attention_softmax(s, table=t, buckets=b, lengths=n, offset=n - 1)
    for i in range(batch):
        row, _ = amd.attention_softmax(s[i:i + 1], table=t, buckets=b, causal=True, offset=int(n[i]) - 1)
        assert torch.equal(row[0], probs[i])


@pytest.mark.parametrize("distance", [3, 16, 129, 1024])
@pytest.mark.parametrize("keys", [50, 300, 3000])
def test_distances(amd, distance, keys):
    """Near and far maps; one that is no order at all, with numbers outside the table."""
    import torch
    s, d, t, b = make(1, 2, 20, keys, 5, "both", buckets=4, distance=distance)
    both_ways(amd, s, d, t, b, offset=keys // 2)
    g = torch.Generator().manual_seed(2)
    b = torch.randint(-2, 9, (2 * distance + 1,), generator=g).to(torch.int32).cuda()
    t = torch.randn((7, 2), generator=g).cuda()
    both_ways(amd, s, d, t, b, offset=keys // 2, p=0.1)
    both_ways(amd, s, d, t, torch.zeros(1, dtype=torch.int32, device="cuda"), offset=-7)     # one bucket for all
    for offset in (-(1 << 39), 1 << 39):
        both_ways(amd, s, d, t, b, offset=offset)


@pytest.mark.parametrize("batch,heads,queries,keys", [(64, 1, 40, 60), (1, 40, 17, 64), (3, 2, 700, 200), (5, 3, 9, 1500)])
def test_table_gradient_over_many_rows(amd, batch, heads, queries, keys):
    both_ways(amd, *make(batch, heads, queries, keys, 6, "both"))
    both_ways(amd, *make(batch, heads, queries, keys, 6, "both"), table_grad=False)


def test_table_gradient_with_less_scratch(amd):
    """Down to none: fewer shares of the rows, the same sums to their rounding."""
    import torch
    s, d, t, b = make(9, 2, 100, 90, 7, "both")
    probs, _ = amd.attention_softmax(s, table=t, buckets=b)
    ref = reference(s, t, b, None, False, 0, 0.0, 0, 0, d)
    desc = amd.AttentionSoftmaxDesc(batch=9, heads=2, queries=100, keys=90, num_buckets=32, max_distance=128)
    full = amd.amsim_attention_softmax_workspace_size(desc)
    assert full > 0
    for nb in (full, full // 2, 2 * 257 * 4, 100, 0):
        ds, dt = torch.empty_like(s), torch.full_like(t, 9.0)
        ws = torch.full((nb + 64,), 0x5A, dtype=torch.uint8, device="cuda")
        amd.amsim_attention_softmax_bwd(desc, d, None, None, probs, None, b, ds, dt, ws, nb)
        near(dt, ref["dt"], ref["dt_tol"], "dtable")
        assert bool((ws[nb:] == 0x5A).all())
    amd.amsim_attention_softmax_bwd(desc, d, None, None, probs, None, b, ds, dt, None, 0)
    near(dt, ref["dt"], ref["dt_tol"], "dtable")


@pytest.mark.parametrize("keys", [9000, 20000, 70000])
def test_long_rows_with_less_scratch(amd, keys):
    """Rows that several blocks share, with room for their sums, for fewer, for none."""
    import torch
    s, d, t, b = make(2, 1, 3, keys, 17, "both")
    probs, _ = amd.attention_softmax(s, table=t, buckets=b)
    ref = reference(s, t, b, None, False, 0, 0.0, 0, 0, d)
    desc = amd.AttentionSoftmaxDesc(batch=2, heads=1, queries=3, keys=keys, num_buckets=32, max_distance=128)
    full = amd.amsim_attention_softmax_workspace_size(desc)
    for nb in (full, full // 2, 3 * 257 * 4, 0):
        ds, dt = torch.empty_like(s), torch.full_like(t, 9.0)
        ws = torch.full((nb + 64,), 0x5A, dtype=torch.uint8, device="cuda")
        amd.amsim_attention_softmax_bwd(desc, d, None, None, probs, None, b, ds, dt, ws, nb)
        near(ds, ref["ds"], ref["ds_tol"], "dscores")
        near(dt, ref["dt"], ref["dt_tol"], "dtable")
        assert bool((ws[nb:] == 0x5A).all())


@pytest.mark.parametrize("ld", [91, 92, 128])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_strides_and_alignment(amd, ld, off):
    """Padded rows, tensors off 16 bytes: within the same bounds as dense ones
    (rows that are not on 16 bytes are added in another order, so equal to the
    bit only among themselves), nothing written behind a row, and in place."""
    import torch
    B, H, Q, K = 2, 3, 11, 90 if ld != 92 else 92
    s, d, t, b = make(B, H, Q, K, 8, "both")

    def place(x):
        buf = torch.full((B * H * Q * ld + 16,), float("nan"), device="cuda")
        v = buf[off:off + B * H * Q * ld].view(B, H, Q, ld)[..., :K]
        if x is not None:
            v.copy_(x)
        return buf, v
    for p in (0.0, 0.2):
        kw = dict(table=t, buckets=b, p=p, seed=3)
        ref = reference(s, t, b, None, False, 0, p, 3, 0, d)
        (_, sp), (_, dp), (obuf, out) = place(s), place(d), place(None)
        probs, stats = amd.attention_softmax(sp, out=out, **kw)
        assert probs is out
        near(probs, ref["probs"], ref["probs"] * ref["E"], "probs")
        assert int(torch.isnan(obuf).sum()) == obuf.numel() - B * H * Q * K
        probs = probs.clone()
        got = amd.attention_softmax_backward(dp, scores=sp, stats=stats, out=out, **kw)
        near(got[0], ref["ds"], ref["ds_tol"], "dscores")
        near(got[1], ref["dt"], ref["dt_tol"], "dtable")
        again = amd.attention_softmax_backward(dp, scores=sp, stats=stats, out=dp, **kw)
        assert again[0] is dp and torch.equal(dp, got[0]) and torch.equal(again[1], got[1])
        amd.attention_softmax(sp, out=sp, **kw)
        assert torch.equal(sp, probs)


def test_empty(amd):
    import torch
    t, b = torch.ones((32, 2), device="cuda"), amd.relative_buckets(32, 128).cuda()
    for shape in ((0, 2, 3, 4), (1, 2, 0, 4), (1, 2, 3, 0)):
        s = torch.zeros(shape, device="cuda")
        probs, stats = amd.attention_softmax(s, table=t, buckets=b)
        assert probs.shape == s.shape and stats.shape == (*shape[:3], 2)
        ds, dt = amd.attention_softmax_backward(s, probs=probs, table=t, buckets=b)
        assert ds.shape == s.shape and not dt.any()


def test_refusals(amd):
    import torch
    s, d, t, b = make(2, 3, 4, 8, 0, "both")
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    probs, stats = amd.attention_softmax(s)
    for bad in (dict(table=t), dict(buckets=b), dict(table=t[:, :2], buckets=b), dict(table=t, buckets=b[:-1]),
                dict(lengths=n[:1]), dict(offset=n[:1])):
        with pytest.raises(ValueError):
            amd.attention_softmax(s, **bad)
    for bad in (dict(lengths=n.long()), dict(offset=n.float()), dict(table=t.double(), buckets=b),
                dict(table=t, buckets=b.long())):
        with pytest.raises(TypeError):
            amd.attention_softmax(s, **bad)
    for x in (s[0], s.transpose(2, 3), s[..., ::2], s[:, :, ::2][:, ::2], s.expand(2, 3, 4, 8)[:, :1].expand(2, 3, 4, 8)):
        with pytest.raises(ValueError):
            amd.attention_softmax(x)
    with pytest.raises(TypeError):
        amd.attention_softmax(s.bfloat16())
    with pytest.raises(ValueError):
        amd.attention_softmax(s, out=probs[:1])
    for bad in (dict(), dict(probs=probs, scores=s, stats=stats), dict(scores=s), dict(probs=probs, p=0.1),
                dict(probs=probs[:1]), dict(scores=s, stats=stats[:1])):
        with pytest.raises(ValueError):
            amd.attention_softmax_backward(d, **bad)
    far = torch.zeros(2 * amd.AMSIM_MAX_DISTANCE + 3, dtype=torch.int32, device="cuda")
    with pytest.raises(amd.AmsimError) as e:
        amd.attention_softmax(s, table=t, buckets=far)
    assert e.value.status == amd.AMSIM_EUNSUPPORTED
    for bad in ((1, 128), (2, 128), (32, 8), (32, 2000)):
        with pytest.raises(ValueError):
            amd.relative_buckets(*bad)


def test_gradient_by_differences(amd):
    """dscores and dtable of a weighted sum of the probabilities (dropped ones
    among them) against central differences.  With steps of h = 2^-5, for the
    largest weight 1: a third derivative of at most 4 / 3 in each of the 6 rows
    that share a bucket leaves 8 h^2 / 6 = 1.3e-3; probabilities within 6e-6 (E
    at A = 6) in 12 rows leave 12 * 4 / 3 * 6e-6 / h = 3.1e-3."""
    import torch
    s, d, t, b = make(1, 2, 6, 9, 9, "both", buckets=8, distance=5)
    kw = dict(buckets=b, p=0.25, seed=8)

    def value(s, t):
        return float((amd.attention_softmax(s, table=t, **kw)[0].double() * d).sum())
    _, stats = amd.attention_softmax(s, table=t, **kw)
    ds, dt = amd.attention_softmax_backward(d, scores=s, stats=stats, table=t, **kw)
    h, size = 2.0 ** -5, float(d.abs().max())
    for x, got in ((s, ds), (t, dt)):
        flat, g = x.view(-1), got.reshape(-1)
        for i in range(0, flat.numel(), 5):
            keep = float(flat[i])
            flat[i] = keep + h
            up = value(s, t)
            flat[i] = keep - h
            down = value(s, t)
            flat[i] = keep
            assert abs((up - down) / (2 * h) - float(g[i])) <= 4.4e-3 * size


def test_streams_and_graphs(amd):
    """Two calls at once on two streams with their own scratch, and a captured
    pair replayed on other inputs."""
    import torch
    jobs = []
    for i in range(2):
        s, d, t, b = make(4, 2, 200, 300, 20 + i, "both")
        kw = dict(table=t, buckets=b, p=0.1, seed=i)
        probs, stats = amd.attention_softmax(s, **kw)
        jobs.append((s, d, kw, probs, stats, amd.attention_softmax_backward(d, scores=s, stats=stats, **kw)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        outs = []
        for st, (s, d, kw, *_) in zip(streams, jobs):
            with torch.cuda.stream(st):
                probs, stats = amd.attention_softmax(s, **kw)
                outs.append((probs, stats, amd.attention_softmax_backward(d, scores=s, stats=stats, **kw)))
        torch.cuda.synchronize()
        for (probs, stats, g), (_, _, _, P, S, G) in zip(outs, jobs):
            assert torch.equal(probs, P) and torch.equal(stats, S) and all(torch.equal(x, y) for x, y in zip(g, G))
    s, d, kw, *_ = jobs[0]
    fixed_s, fixed_d, step = s.clone(), d.clone(), torch.zeros(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        probs, stats = amd.attention_softmax(fixed_s, step=step, **kw)
        ds, dt = amd.attention_softmax_backward(fixed_d, scores=fixed_s, stats=stats, step=step, **kw)
    for i, (s, d, *_) in enumerate(jobs):
        fixed_s.copy_(s)
        fixed_d.copy_(d)
        step.fill_(i)
        graph.replay()
        P, S = amd.attention_softmax(s, call=i, **kw)
        G = amd.attention_softmax_backward(d, scores=s, stats=S, call=i, **kw)
        assert torch.equal(probs, P) and torch.equal(ds, G[0]) and torch.equal(dt, G[1])
