"""The exact operators at their edges: tensors whose ends are off 16 bytes, empty
batches, non-finite and masked inputs, calls from several threads."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", range(8))
@pytest.mark.parametrize("cols", [1017, 1020])
def test_streamed_ends_off_16_bytes(amd, off, cols):
    """Streamed rows whose tensor starts `off` elements past 16 bytes, NaN right
    before its first element and behind its last: every row, the first and the
    last among them, as in a call of those rows alone (loaded directly)."""
    import torch
    rows = 2500
    g = torch.Generator(device="cuda").manual_seed(off)

    def place(dtype):
        buf = torch.full((rows * cols + 16,), float("nan"), dtype=dtype, device="cuda")
        v = buf[off:off + rows * cols].view(rows, cols)
        v.copy_(torch.randn((rows, cols), generator=g, device="cuda"))
        return v
    x, y, dr, dn = place(torch.bfloat16), place(torch.float32), place(torch.bfloat16), place(torch.bfloat16)
    w, v = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda") for _ in range(2))
    kw = dict(alpha=0.5)
    fwd = amd.block_norm(x, y, w, v, n_dtype=torch.bfloat16, **kw)
    ro = place(torch.bfloat16)
    ro.copy_(fwd[0])
    back = amd.block_norm_backward(dr, dn, ro, y, w, v, fwd[2], fwd[3], **kw)
    assert all(bool(torch.isfinite(t).all()) for t in fwd + tuple(t for t in back if t is not None))
    for s in (slice(0, 2), slice(rows - 2, rows)):
        few = amd.block_norm(x[s], y[s], w, v, n_dtype=torch.bfloat16, **kw)
        assert all(torch.equal(p[s], q) for p, q in zip(fwd, few))
        few = amd.block_norm_backward(dr[s], dn[s], ro[s], y[s], w, v, fwd[2][s], fwd[3][s], **kw)
        assert torch.equal(back[0][s], few[0]) and torch.equal(back[1][s], few[1])
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)


@pytest.mark.parametrize("groups", [1, 3])
def test_empty_batch_has_a_zero_gate_gradient(amd, groups):
    """Every sum over no rows is zero, whatever the memory held before."""
    import torch
    f = dict(device="cuda")
    x, w, gate = torch.empty((0, 24), **f), torch.ones(24, **f), torch.ones((groups, 24), **f)
    for _ in range(3):
        torch.full((4096,), float("nan"), **f)               # what the allocator hands out next
        r, n, post, pre = amd.block_norm(x, x, w, w, gate=gate)
        assert r.shape == n.shape == (0, 24)
        for t in amd.block_norm_backward(x, x, r, x, w, w, post, pre, gate=gate)[2:]:
            assert not t.any()
    d = amd.BlockNormDesc(rows=0, cols=24, alpha=1.0)
    sums = [torch.full((24,), 3.0, **f) for _ in range(3)]
    amd.amsim_block_norm_bwd(d, x, x, x, x, gate, w, w, post, pre, x, x, *sums)
    assert not torch.stack(sums).any()


def test_layer_on_an_empty_batch(amd):
    import torch
    from approximate_multiplier_dnn_gb300.layers import BlockNorm
    norm = BlockNorm(24, gate="channel")
    r, n = norm(torch.zeros((0, 5, 24), device="cuda"), torch.zeros((0, 5, 24), device="cuda"))
    assert r.shape == n.shape == (0, 5, 24)
    (r.sum() + n.sum()).backward()
    assert not torch.stack([norm.gate.grad[0], norm.w_post.grad, norm.w_pre.grad]).any()


def test_threads_with_different_widths(amd):
    """Host threads that launch one kernel with different amounts of shared
    memory at once: every call launches, and leaves what a call by itself does."""
    import ctypes
    import threading

    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    fn, start, failed = amd.lib().amsim_block_norm_fwd, threading.Barrier(8), []

    def job(rows, cols):
        x, y = (torch.randn((rows, cols), generator=g, device="cuda") for _ in range(2))
        w = torch.ones(cols, device="cuda")
        want = amd.block_norm(x, y, w, w)
        out = [torch.zeros_like(t) for t in want]
        d = amd.BlockNormDesc(rows=rows, cols=cols, alpha=1.0, eps=1e-6)
        stream = torch.cuda.Stream()
        args = [ctypes.byref(d)] + [t.data_ptr() if t is not None else None for t in (x, y, None, w, w, *out)]
        args.append(stream.cuda_stream)

        def run():
            start.wait()
            failed.extend(rc for rc in (fn(*args) for _ in range(4000)) if rc)
        return run, want, out, (x, y, w, d, stream)
    jobs = [job(rows, cols) for rows, cols in ((160, 4096), (320, 2048), (160, 3584), (320, 1800)) for _ in range(2)]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=j[0]) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, f"{len(failed)} calls failed: {sorted(set(failed))}"
    for _, want, out, _ in jobs:
        assert all(torch.equal(p, q) for p, q in zip(out, want))


def vocab_inputs(tokens, vocab, dim, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    h = torch.randn((tokens, dim), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((vocab, dim), generator=g) * 2 / dim ** 0.5).to(torch.bfloat16).cuda()
    return h, w, torch.randint(0, vocab, (tokens,), generator=g).cuda()


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("tokens,vocab,dim", [(60, 500, 64), (300, 1000, 130)])
def test_non_finite_hidden_state_gives_nan_gradients(amd, value, tokens, vocab, dim):
    """A token that counts and has a non-finite hidden state has a NaN loss: its
    gradient is NaN, and dw, to which it adds, not one that could be taken for
    a token's."""
    import torch
    h, w, t = vocab_inputs(tokens, vocab, dim)
    clean = amd.vocab_loss_grad(h, w, t)
    h[7, 5] = float(value)
    loss, row, lse, dh, dw = amd.vocab_loss_grad(h, w, t)
    assert bool(torch.isnan(torch.stack([loss[0], row[7], lse[7]])).all())
    assert bool(torch.isnan(dh[7]).all()) and bool(torch.isnan(dw).all())
    keep = [i for i in range(tokens) if i != 7]
    assert torch.equal(dh[keep], clean[3][keep]) and torch.equal(row[keep], clean[1][keep])


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("tokens,vocab,dim", [(60, 500, 64), (300, 1000, 130), (1100, 700, 2100)])
def test_ignored_tokens_add_nothing(amd, value, tokens, vocab, dim):
    """Tokens without a target, or with one outside the vocabulary, add nothing
    to dh and dw, whatever their hidden states hold (padding, say)."""
    import torch
    h, w, t = vocab_inputs(tokens, vocab, dim, seed=1)
    t[3::5] = -100
    t[11] = vocab
    want = amd.vocab_loss_grad(h, w, t)
    h[3::5, ::2] = float(value)
    h[11] = float(value)
    loss, row, lse, dh, dw = amd.vocab_loss_grad(h, w, t)
    assert torch.equal(dh, want[3]) and torch.equal(dw, want[4])
    assert not dh[3::5].any() and not dh[11].any() and bool(torch.isfinite(dw).all())
    t[11] = -100
    assert bool(torch.isfinite(amd.vocab_loss_grad(h, w, t)[0]).all())


@pytest.mark.parametrize("tokens", [1000, 5000])
def test_infinite_row_loss_makes_the_loss_infinite(amd, tokens):
    """A target with probability zero costs infinity, and so does the batch,
    however many other tokens are added to it."""
    import torch
    h, w, t = vocab_inputs(tokens, 100, 16, seed=2)
    h[:, 0] = 1.0
    w[37, 0] = float("-inf")                                # no token can be 37
    t[t == 37] = 36
    assert bool(torch.isfinite(amd.vocab_loss(h, w, t)[0]))
    t[5] = t[tokens - 7] = 37
    loss, row, lse = amd.vocab_loss(h, w, t)
    assert bool(torch.isposinf(row[5])) and bool(torch.isfinite(lse).all())
    assert bool(torch.isposinf(loss))


def test_evaluation_scratch_is_small(amd):
    """Aligned operands are not copied, and take no scratch for copies: the loss
    alone needs far less than a copy of w."""
    import torch
    h, w, t = vocab_inputs(256, 65536, 512, seed=3)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    amd.vocab_loss(h, w, t)
    assert torch.cuda.max_memory_allocated() - before < 4 << 20        # w: 64 MiB


def test_head_evaluation_launches_the_loss_alone(amd):
    """Two kernels (the logits' product and the merge) and the same value."""
    import torch
    from approximate_multiplier_dnn_gb300.layers import VocabHead
    h, _, t = vocab_inputs(64, 500, 64)
    head = VocabHead(64, 500, generator=torch.Generator().manual_seed(0))
    train = head(h, t).detach()
    before = amd.amsim_kernel_launches()
    with torch.no_grad():
        loss = head(h, t)
    assert amd.amsim_kernel_launches() - before == 2
    assert torch.equal(loss, train) and not loss.requires_grad


@pytest.mark.parametrize("factor", [1 / 3, 0.01])
def test_upstream_factor_is_not_rounded(amd, factor):
    """Gradients of the head scaled by an fp32 factor that bf16 does not hold, to the bit."""
    import torch
    from approximate_multiplier_dnn_gb300.layers import VocabHead
    h, _, t = vocab_inputs(100, 300, 40, seed=4)
    head = VocabHead(40, 300, generator=torch.Generator().manual_seed(1))
    loss = head(h.requires_grad_(), t)
    _, _, _, dh, dw = amd.vocab_loss_grad(h.detach(), head.weight.detach(), t)
    (loss * factor).backward()
    f = torch.tensor(factor, dtype=torch.float32, device="cuda")
    assert torch.equal(h.grad, (dh.float() * f).to(torch.bfloat16))
    assert torch.equal(head.weight.grad, (dw.float() * f).to(torch.bfloat16))


@pytest.mark.parametrize("used", ["r", "n"])
@pytest.mark.parametrize("first", [False, True])
def test_layer_with_an_unused_output(amd, used, first):
    """Gradients through one output of BlockNorm are those with zeros for the
    other's, to the bit."""
    import torch
    from approximate_multiplier_dnn_gb300.layers import BlockNorm
    g = torch.Generator(device="cuda").manual_seed(5)
    x, y, c = (torch.randn((30, 48), generator=g, device="cuda") for _ in range(3))
    norm = BlockNorm(48, gate=None if first else "channel")
    leaves = [x.requires_grad_(), *([] if first else [y.requires_grad_()]), *norm.parameters()]
    out = norm(x) if first else norm(x, y)
    got = torch.autograd.grad((out[used == "n"] * c).sum(), leaves, allow_unused=True)
    out = norm(x) if first else norm(x, y)
    want = torch.autograd.grad((out[used == "n"] * c).sum() + (out[used == "r"] * 0).sum(), leaves, allow_unused=True)
    for p, q in zip(got, want):
        assert (p is None) == (q is None) and (p is None or torch.equal(p, q))


@pytest.mark.parametrize("drop", ["dr", "dn"])
@pytest.mark.parametrize("rows,cols", [(2600, 512), (640, 3047), (308, 8191), (308, 8192), (2440, 1013), (2440, 1012)])
@pytest.mark.parametrize("x,n", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float32", "bfloat16")])
def test_streamed_backward_without_a_gradient(amd, drop, rows, cols, x, n):
    """A gradient that is not there is one of zeros: dx and dy to the bit, the
    sums over rows up to the order of their terms (two sums of R terms, each
    within R + 64 u of the sum of magnitudes); without y as well."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(cols)
    X, N = getattr(torch, x), getattr(torch, n)
    a, y, dr, dn = (torch.randn((rows, cols), generator=g, device="cuda").to(t) for t in (X, N, X, N))
    w, v = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda") for _ in range(2))
    gate = torch.rand((2, cols), generator=g, device="cuda")
    r, _, post, pre = amd.block_norm(a, y, w, v, gate=gate, n_dtype=N)
    want = amd.block_norm_backward(dr * (drop != "dr"), dn * (drop != "dn"), r, y, w, v, post, pre, gate=gate)
    got = amd.block_norm_backward(None if drop == "dr" else dr, None if drop == "dn" else dn, r, y, w, v, post, pre,
                                  gate=gate)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    yh, rh = (y.double() * post[:, None]).abs(), (r.double() * pre[:, None]).abs()
    u = got[0].double().abs() * yh * 1.01                    # dx as the sums take it, before its rounding
    mags = [(u * w).view(2, rows // 2, cols).sum(1), (u.view(2, rows // 2, cols) * gate[:, None]).sum((0, 1)),
            (dn.double().abs() * rh).sum(0)]
    for p, q, mag in zip(got[2:], want[2:], mags):
        assert bool(((p.double() - q.double()).abs() <= 2 * (rows + 64) * 2.0 ** -24 * mag).all())
    if drop == "dr":                                          # neither y nor a gradient of r
        dx, _, _, _, dw = amd.block_norm_backward(None, dn, r, None, None, v, None, pre)
        assert torch.equal(dx, want[0])
        assert bool(((dw.double() - want[4].double()).abs() <= 2 * (rows + 64) * 2.0 ** -24 * mags[2]).all())
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_follows_loaded_weights(amd, bits):
    """Weights loaded into the head between steps stay (their gradients are
    zero and decay is off), and a step's own writes are not taken for a load."""
    import torch
    from approximate_multiplier_dnn_gb300.layers import VocabHead
    from approximate_multiplier_dnn_gb300.optim import AdamW
    head, other = (VocabHead(40, 300, generator=torch.Generator().manual_seed(i)) for i in (1, 2))
    opt = AdamW(head.parameters(), lr=1e-2, weight_decay=0.0, moment_bits=bits)
    w = head.weight
    for _ in range(3):
        w.grad = torch.randn_like(w)
        opt.step()
        master = opt.state[w]["master"]
        assert torch.equal(w.detach().view(-1), master.to(torch.bfloat16)) and not torch.equal(w.float().view(-1), master)
    old, new = w.detach().clone().view(-1), other.weight.detach().view(-1)
    master = opt.state[w]["master"].clone()
    head.load_state_dict(other.state_dict())
    opt.param_groups[0]["lr"] = 0.0
    opt.step()
    assert torch.equal(w, other.weight)
    assert torch.equal(opt.state[w]["master"], torch.where(old == new, master, new.float()))   # low bits stay where it does


def test_optimizer_with_late_gradients(amd):
    """A parameter that joins at step 40 moves as in an optimizer of its own, to the bit."""
    import torch
    from approximate_multiplier_dnn_gb300.optim import AdamW
    g = torch.Generator(device="cuda").manual_seed(0)
    a, b = (torch.nn.Parameter(torch.randn(n, generator=g, device="cuda")) for n in (1000, 777))
    c = torch.nn.Parameter(b.detach().clone())
    both, alone = AdamW([a, b]), AdamW([c])
    for i in range(45):
        a.grad = torch.randn(a.shape, generator=g, device="cuda")
        if i >= 40:
            b.grad = torch.randn(b.shape, generator=g, device="cuda")
            c.grad = b.grad.clone()
            alone.step()
        both.step()
    assert torch.equal(b, c) and both.state[b]["step"] == 5 and both.state[a]["step"] == 45


@pytest.mark.parametrize("cols,ld,off", [(1024, 1024, 0), (1024, 1040, 8), (1016, 1019, 3), (1013, 1013, 1)])
@pytest.mark.parametrize("groups", [1, 4])
def test_streamed_in_place_with_strides(amd, cols, ld, off, groups):
    """Streamed rows with a stride, r over x and n over y, dx over dr and dy over
    dn: what the same layout gives beside its inputs, to the bit, and nothing
    between the rows is written."""
    import torch
    rows, B = 2500, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(cols)

    def place(t=None):
        buf = torch.full((rows * ld + off + 8,), 5.0, dtype=B, device="cuda")
        v = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
        v.copy_(torch.randn((rows, cols), generator=g, device="cuda") if t is None else t)
        return buf, v
    w, v = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda") for _ in range(2))
    gate = torch.rand((groups, cols), generator=g, device="cuda")
    d = amd.BlockNormDesc(rows=rows, cols=cols, gate_rows=rows // groups, alpha=0.5, eps=1e-6, x_type=1, y_type=1,
                          n_type=1, ldx=ld, ldy=ld, ldr=ld, ldn=ld, lddr=ld, lddn=ld, lddx=ld, lddy=ld)
    (xb, x), (yb, y), (_, r), (_, n) = (place() for _ in range(4))
    post, pre = (torch.empty(rows, device="cuda") for _ in range(2))
    y0 = place(y)[1]
    amd.amsim_block_norm_fwd(d, x, y, gate, w, v, r, n, post, pre)
    amd.amsim_block_norm_fwd(d, x, y, gate, w, v, x, y, post, pre)
    assert torch.equal(x, r) and torch.equal(y, n)
    (drb, dr), (dnb, dn), (_, dx), (_, dy) = (place() for _ in range(4))
    ws = amd.workspace(amd.amsim_block_norm_workspace_size(d))
    sums = [[torch.empty_like(t) for t in (gate, w, v)] for _ in range(2)]
    amd.amsim_block_norm_bwd(d, dr, dn, r, y0, gate, w, v, post, pre, dx, dy, *sums[0], ws=ws)
    amd.amsim_block_norm_bwd(d, dr, dn, r, y0, gate, w, v, post, pre, dr, dn, *sums[1], ws=ws)
    assert torch.equal(dr, dx) and torch.equal(dn, dy) and all(torch.equal(p, q) for p, q in zip(*sums))
    for buf, t in ((xb, x), (yb, y), (drb, dr), (dnb, dn)):
        t.fill_(5.0)
        assert bool((buf == 5.0).all())
    assert amd.amsim_device_errors() == (amd.AMSIM_OK, 0)
