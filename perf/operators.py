"""The exact (IEEE) operators of a language model's training step, as measured cases.

Three operators stand beside the approximate contractions of a training step:

norm    the block norm: the norms before and after a block, fused with the
        block's gate and the residual scale (forward and backward);
vocab   the vocabulary loss: softmax cross entropy of h W^T against token
        targets without keeping the logits, with the gradients of h and W;
adamw   one AdamW step over many tensors, moments in 32 bits or in 8.

With ``own`` false a case runs in its plain form, elementary torch operations
in fp32 rounded once at the end; with ``own`` true it calls the package.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
IGNORE = -100
EPS = 1e-6
ALPHA = 0.5          # residual scale of the block norm
LR, WD, BETA1, BETA2, ADAM_EPS = 3e-4, 0.1, 0.9, 0.999, 1e-8
BLOCK = 256          # elements that share one scale of an 8-bit moment


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token through one block of a small model: latency alone
        _norm("norm_fwd_token", "fwd", 1, 1024, "f32", "f32", "f32", 1),
        # a training batch, bf16 residual stream, a gate for each of 8 sequences
        _norm("norm_fwd_batch", "fwd", 16384, 4096, "bf16", "bf16", "bf16", 8),
        # an odd number of tokens at the width of the framework's MLP, all fp32
        _norm("norm_bwd_odd", "bwd", 4099, 1000, "f32", "f32", "f32", 1),
        # a training batch: fp32 residual stream, bf16 at the block's edges
        _norm("norm_bwd_batch", "bwd", 16384, 2048, "f32", "bf16", "bf16", 4),
        # the last tokens of a short batch against a small vocabulary
        _vocab("vocab_grad_few", True, 24, 8192, 256, 0.0),
        # perplexity of a batch: the loss alone
        _vocab("vocab_loss_eval", False, 4096, 32768, 1024, 0.0),
        # packed prompts: a third of the tokens carry no target, no size is round
        _vocab("vocab_grad_odd", True, 1531, 50021, 1000, 0.33),
        # a training batch of 8 x 1024 tokens
        _vocab("vocab_grad_batch", True, 8192, 65536, 4096, 0.05),
        # as many parameters as the MLP 784-1000-500-10 with its biases
        _adamw("adamw_mlp", 32, "f32", False, 1_290_510, 6),
        # a model of some hundred tensors, moments in fp32, bf16 copies for the next pass
        _adamw("adamw_model", 32, "f32", True, 256_000_000, 200),
        # small odd tensors, as of many adapters, moments in 8 bits
        _adamw("adamw8_small", 8, "f32", False, 700_001, 90),
        # the model again with bf16 gradients, moments in 8 bits
        _adamw("adamw8_model", 8, "bf16", True, 256_000_000, 200),
    ]


def _norm(name, way, rows, cols, x, y, n, groups):
    return {"name": name, "op": "norm", "way": way, "rows": rows, "cols": cols, "x": x, "y": y, "n": n,
            "groups": groups}


def _vocab(name, grad, tokens, vocab, dim, ignored):
    return {"name": name, "op": "vocab", "grad": grad, "tokens": tokens, "vocab": vocab, "dim": dim,
            "ignored": ignored}


def _adamw(name, bits, g, copy, total, tensors):
    return {"name": name, "op": "adamw", "bits": bits, "g": g, "copy": copy, "total": total, "tensors": tensors}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "vocab", "adamw"))
    if op == "norm":
        cols = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            cols = -(-cols // 8) * 8             # most models' widths are multiples of 8, some are not
        rows = _log(rng, 1, min(16384, 16384 * 4096 // cols))
        groups = rng.choice((1, 1, 2, 5)) if rows >= 16 else 1
        c = _norm("", rng.choice(("fwd", "bwd")), rows - rows % groups, cols, rng.choice(("f32", "bf16")),
                  rng.choice(("f32", "bf16")), rng.choice(("f32", "bf16")), groups)
    elif op == "vocab":
        dim = _log(rng, 64, 4096)
        if rng.random() < 0.8:
            dim = -(-dim // 8) * 8
        vocab = _log(rng, 1000, 131072)
        tokens = _log(rng, 1, max(1, min(8192, 8192 * 65536 * 4096 // (vocab * dim))))
        c = _vocab("", rng.random() < 0.7, tokens, vocab, dim, rng.choice((0.0, 0.1, 0.5)))
    else:
        total = _log(rng, 10_000, 256_000_000)
        c = _adamw("", rng.choice((8, 32)), rng.choice(("f32", "bf16")), rng.random() < 0.5, total,
                   min(_log(rng, 1, 400), max(1, total // 1000)))
    del c["name"]
    return c


def work(case):
    if case["op"] == "norm":
        e, v = case["rows"] * case["cols"], 4 * case["cols"]
        x, y, n = SIZE[case["x"]], SIZE[case["y"]], SIZE[case["n"]]
        if case["way"] == "fwd":                 # x, y in; the new stream and the next block's input out
            return {"bytes": e * (2 * x + y + n) + v * (2 + case["groups"]) + 8 * case["rows"], "flops": 10 * e}
        # y, r, dr, dn in; dx, dy out
        return {"bytes": e * (3 * x + 2 * y + n) + 2 * v * (2 + case["groups"]) + 8 * case["rows"], "flops": 24 * e}
    if case["op"] == "vocab":
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        both = 2 * (t + v) * d
        return {"bytes": both * (2 if case["grad"] else 1) + 20 * t, "flops": (6 if case["grad"] else 2) * t * v * d}
    n, g = case["total"], SIZE[case["g"]]
    # parameter in and out, gradient in, both moments in and out; 8-bit moments also out as values
    moments = 16 if case["bits"] == 32 else 4 + 8 + 16 / BLOCK
    return {"bytes": n * (8 + g + moments + (2 if case["copy"] else 0)), "flops": 15 * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _sizes(case):
    """Tensor sizes of a model: a few large matrices, many small vectors, most of them odd."""
    n, total = case["tensors"], case["total"]
    share = [1.0 / (1 + (7 * i) % n) for i in range(n)]
    s = [max(1, int(total * x / sum(share))) for x in share]
    s[0] += total - sum(s)
    return s


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    if case["op"] == "norm":
        R, C = case["rows"], case["cols"]
        X, Y, N = TYPES[case["x"]], TYPES[case["y"]], TYPES[case["n"]]
        y = (_randn(g, R, C) * 1.3).to(Y)
        x = (_randn(g, R, C) * 2.0).to(X)
        st.update(y=y, w_post=1.0 + 0.1 * _randn(g, C), w_pre=1.0 + 0.1 * _randn(g, C),
                  gate=0.5 + 0.2 * _randn(g, case["groups"], C), n_type=N)
        if case["way"] == "fwd":
            st["x"] = x
        else:                                    # the forward's outputs, as it left them, and the gradients
            r, _, st["rstd_post"], st["rstd_pre"] = _norm_fwd_plain(dict(st, x=x))
            st.update(r=r, dr=(0.01 * _randn(g, R, C)).to(X), dn=(0.01 * _randn(g, R, C)).to(N))
    elif case["op"] == "vocab":
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        st["h"] = _randn(g, T, D).to(torch.bfloat16)
        st["w"] = (_randn(g, V, D) * (2.0 / math.sqrt(D))).to(torch.bfloat16)
        u = torch.rand(T, generator=g, device="cuda")
        t = (u * u * u * V).long().clamp_(max=V - 1)         # frequent tokens first
        gone = torch.rand(T, generator=g, device="cuda") < case["ignored"]
        st["targets"] = torch.where(gone, torch.full_like(t, IGNORE), t)
    else:
        sizes = _sizes(case)
        starts, at = [], 0
        for s in sizes:                          # one buffer; each tensor starts on a block of its own
            starts.append(at)
            at += -(-s // BLOCK) * BLOCK
        used = torch.zeros(at, dtype=torch.bool, device="cuda")
        for a, s in zip(starts, sizes):
            used[a:a + s] = True
        st["p"] = _randn(g, at).mul_(0.02).mul_(used)
        st["grad"] = _randn(g, at).mul_(1e-3).mul_(used).to(TYPES[case["g"]])
        st["scale"] = torch.full((1,), 0.7, device="cuda")   # of clipping the gradient's norm
        st["copy"] = torch.zeros(at, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
        m = _randn(g, at).mul_(3e-4).mul_(used)
        v = _randn(g, at).square_().mul_(1e-6).mul_(used)
        if case["bits"] == 32:
            st["m"], st["v"] = m, v
        else:
            st["m"], st["m_scale"] = _encode(m, True)
            st["v"], st["v_scale"] = _encode(v, False)
        st["step"] = 100
        st["spans"] = list(zip(starts, sizes))
        if own:                                  # the table of tensors that an optimizer keeps
            import approximate_multiplier_dnn_gb300 as am
            st["table"] = am.adamw_table([_tensor(am, st, a, s) for a, s in st["spans"]])
    return st


def _tensor(am, st, a, s):
    b, nb = a // BLOCK, -(-s // BLOCK)
    eight = st["case"]["bits"] == 8
    return am.AdamwTensor.make(st["p"][a:a + s], st["grad"][a:a + s], st["m"][a:a + s], st["v"][a:a + s],
                               m_scale=st["m_scale"][b:b + nb] if eight else None,
                               v_scale=st["v_scale"][b:b + nb] if eight else None,
                               copy=st["copy"][a:a + s] if st["copy"] is not None else None, weight_decay=WD)


# ------------------------------------------------------------------ plain forms
def _rms(t):
    return torch.rsqrt(t.square().mean(1, keepdim=True) + EPS)


def _gate_rows(st, rows):
    return st["gate"].repeat_interleave(rows // st["gate"].shape[0], 0)


def _norm_fwd_plain(st):
    x, y = st["x"].float(), st["y"].float()
    rstd_post = _rms(y)
    r = x + ALPHA * _gate_rows(st, x.shape[0]) * (y * rstd_post * st["w_post"])
    rstd_pre = _rms(r)
    n = r * rstd_pre * st["w_pre"]
    return r.to(st["x"].dtype), n.to(st["n_type"]), rstd_post[:, 0], rstd_pre[:, 0]


def _norm_bwd_plain(st):
    y, r, dr, dn = (st[k].float() for k in ("y", "r", "dr", "dn"))
    groups, (rows, cols) = st["gate"].shape[0], y.shape
    rhat = r * st["rstd_pre"][:, None]
    t = dn * st["w_pre"]
    dx = dr + st["rstd_pre"][:, None] * (t - rhat * (t * rhat).mean(1, keepdim=True))
    yhat = y * st["rstd_post"][:, None]
    du = ALPHA * _gate_rows(st, rows) * dx
    dgate = (ALPHA * dx * (yhat * st["w_post"])).view(groups, rows // groups, cols).sum(1)
    s = du * st["w_post"]
    dy = st["rstd_post"][:, None] * (s - yhat * (s * yhat).mean(1, keepdim=True))
    return (dx.to(st["r"].dtype), dy.to(st["y"].dtype), dgate, (du * yhat).sum(0), (dn * rhat).sum(0))


def _vocab_plain(st):
    h, w, t = st["h"].float(), st["w"].float(), st["targets"]
    valid = t != IGNORE
    at = torch.where(valid, t, torch.zeros_like(t))[:, None]
    logits = h @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = top + (logits - top).exp().sum(1, keepdim=True).log()
    row = torch.where(valid, (lse - logits.gather(1, at))[:, 0], torch.zeros_like(lse[:, 0]))
    share = valid / valid.sum().clamp(min=1)
    loss = (row * share).sum().reshape(1)
    if not st["case"]["grad"]:
        return loss, row, lse[:, 0]
    g = (logits - lse).exp_()
    g.scatter_add_(1, at, torch.full_like(lse, -1.0))
    g *= share[:, None]
    return loss, row, lse[:, 0], (g @ w).to(torch.bfloat16), (g.t() @ h).to(torch.bfloat16)


def _encode(x, signed):
    """8-bit codes and block scales of a moment: the square (first moment) or
    fourth (second) power of code / top, times the block's largest magnitude."""
    b = x.view(-1, BLOCK)
    scale = b.abs().amax(1)
    top = torch.full_like(scale, 127.0 if signed else 255.0)
    root = scale.sqrt() if signed else scale.sqrt().sqrt()
    k = torch.where(root > 0, top / root, torch.zeros_like(root))
    f = b.abs().sqrt() if signed else b.sqrt().sqrt()
    q = torch.minimum((f * k[:, None]).round(), top[:, None])
    if signed:
        q = torch.where(b < 0, -q, q).to(torch.int8)
    else:                                        # a second moment above zero stays above zero
        q = torch.where(b > 0, q.clamp(min=1.0), q).to(torch.uint8)
    return q.view(-1), scale


def _decode(q, scale, signed):
    t = q.view(-1, BLOCK).float() * (1.0 / 127.0 if signed else 1.0 / 255.0)
    t2 = t * t.abs()
    return ((t2 if signed else t2 * t2) * scale[:, None]).view(-1)


def _adamw_plain(st):
    eight = st["case"]["bits"] == 8
    t = st["step"]
    g = st["grad"].float() * st["scale"]
    m = _decode(st["m"], st["m_scale"], True) if eight else st["m"]
    v = _decode(st["v"], st["v_scale"], False) if eight else st["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    step = m / (v.sqrt() * (1.0 / math.sqrt(1.0 - BETA2 ** t)) + ADAM_EPS)
    st["p"].copy_(st["p"] * (1.0 - LR * WD) - step * (LR / (1.0 - BETA1 ** t)))
    if st["copy"] is not None:
        st["copy"].copy_(st["p"])
    if eight:
        for name, x, signed in (("m", m, True), ("v", v, False)):
            q, scale = _encode(x, signed)
            st[name].copy_(q)
            st[name + "_scale"].copy_(scale)
        m, v = _decode(st["m"], st["m_scale"], True), _decode(st["v"], st["v_scale"], False)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return m, v


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if op == "norm":
        fwd = st["case"]["way"] == "fwd"
        if not own:
            return _norm_fwd_plain(st) if fwd else _norm_bwd_plain(st)
        import approximate_multiplier_dnn_gb300 as am
        if fwd:
            return am.block_norm(st["x"], st["y"], st["w_post"], st["w_pre"], gate=st["gate"], alpha=ALPHA, eps=EPS,
                                 n_dtype=st["n_type"])
        return am.block_norm_backward(st["dr"], st["dn"], st["r"], st["y"], st["w_post"], st["w_pre"],
                                      st["rstd_post"], st["rstd_pre"], gate=st["gate"], alpha=ALPHA)
    if op == "vocab":
        if not own:
            return _vocab_plain(st)
        import approximate_multiplier_dnn_gb300 as am
        if st["case"]["grad"]:
            return am.vocab_loss_grad(st["h"], st["w"], st["targets"], ignore_index=IGNORE)
        return am.vocab_loss(st["h"], st["w"], st["targets"], ignore_index=IGNORE)
    if own:
        import approximate_multiplier_dnn_gb300 as am
        am.adamw_step(st["table"], lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, step=st["step"],
                      grad_scale=st["scale"])
        if st["case"]["bits"] == 8:              # the moments' values, as a checkpoint writes them
            m = am.adamw_moment_values(st["m"], st["m_scale"])
            v = am.adamw_moment_values(st["v"], st["v_scale"])
        else:
            m, v = st["m"], st["v"]
    else:
        m, v = _adamw_plain(st)
    st["step"] += 1
    return st["p"], m, v, st["copy"]


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] == "vocab" and (6 if case["grad"] else 2) * case["tokens"] * case["vocab"] * case["dim"] > 1.4e13:
        return None                              # over 20 seconds at the card's fp64 rate
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_fwd_exact(st) if case["way"] == "fwd" else _norm_bwd_exact(st)
    return _vocab_exact(st) if case["op"] == "vocab" else _adamw_exact(st)


def _norm_fwd_exact(st):
    x, y = st["x"].double(), st["y"].double()
    C = x.shape[1]
    gate = st["gate"].double().unsqueeze(1).expand(-1, x.shape[0] // st["gate"].shape[0], C).reshape(-1, C)
    post = (torch.einsum("rc,rc->r", y, y) / C + EPS).pow(-0.5)
    r = x + ALPHA * gate * st["w_post"].double() * torch.einsum("rc,r->rc", y, post)
    pre = (torch.einsum("rc,rc->r", r, r) / C + EPS).pow(-0.5)
    return r, torch.einsum("rc,r,c->rc", r, pre, st["w_pre"].double()), post, pre


def _norm_bwd_exact(st):
    """By differentiating the definition, with the forward's saved factors as they are:
    d(rstd)/d(row) = -rstd^3 row / C."""
    y, r, dr, dn = (st[k].double() for k in ("y", "r", "dr", "dn"))
    a, b = st["rstd_pre"].double(), st["rstd_post"].double()
    wp, wq = st["w_post"].double(), st["w_pre"].double()
    R, C = y.shape
    gate = st["gate"].double().unsqueeze(1).expand(-1, R // st["gate"].shape[0], C).reshape(-1, C)
    d_a = (dn * wq * r).sum(1)
    dx = dr + dn * wq * a[:, None] - r * (d_a * a.pow(3) / C)[:, None]
    z = y * wp                                   # the block's output up to its row factor
    dz = ALPHA * gate * dx
    d_b = (dz * z).sum(1)
    dy = dz * wp * b[:, None] - y * (d_b * b.pow(3) / C)[:, None]
    dgate = torch.stack([(ALPHA * dx[k] * z[k] * b[k, None]).sum(0)
                         for k in torch.arange(R, device=y.device).chunk(st["gate"].shape[0])])
    return dx, dy, dgate, (dz * y * b[:, None]).sum(0), (dn * r * a[:, None]).sum(0)


def _vocab_exact(st):
    h, w, t = st["h"].double(), st["w"].double(), st["targets"]
    T, V = h.shape[0], w.shape[0]
    count = int((t != IGNORE).sum())
    row = torch.zeros(T, dtype=torch.float64, device=h.device)
    lse, dh, dw = torch.zeros_like(row), torch.zeros_like(h), torch.zeros_like(w)
    step = max(1, 2_000_000_000 // (8 * V))
    for a in range(0, T, step):                  # some rows at a time
        s = slice(a, a + step)
        z = h[s] @ w.t()
        lse[s] = torch.logsumexp(z, 1)
        rows = torch.nonzero(t[s] != IGNORE)[:, 0]
        cols = t[s][rows]
        row[a + rows] = lse[s][rows] - z[rows, cols]
        if st["case"]["grad"]:
            p = torch.zeros_like(z)
            p[rows] = torch.exp(z[rows] - lse[s][rows, None])
            p[rows, cols] -= 1.0
            p /= max(count, 1)
            dh[s] = p @ w
            dw += p.t() @ h[s]
    loss = (row.sum() / max(count, 1)).reshape(1)
    return (loss, row, lse, dh, dw) if st["case"]["grad"] else (loss, row, lse)


def _adamw_exact(st):
    eight = st["case"]["bits"] == 8
    t = st["step"]

    def values(name, power, top):
        if not eight:
            return st[name].double()
        q = st[name].double().view(-1, BLOCK) / top
        return (q.sign() * q.abs().pow(power) * st[name + "_scale"].double()[:, None]).view(-1)

    def stored(x, power, top):
        if not eight:
            return x
        b = x.view(-1, BLOCK)
        scale = b.abs().amax(1, keepdim=True)
        q = torch.nan_to_num((b.abs() / scale).pow(1.0 / power)).mul(top).round()
        if power == 4:
            q = torch.where(b > 0, q.clamp(min=1.0), q)
        return (b.sign() * (q / top).pow(power) * scale).view(-1)

    g = st["grad"].double() * st["scale"].double()
    m = BETA1 * values("m", 2, 127.0) + (1.0 - BETA1) * g
    v = BETA2 * values("v", 4, 255.0) + (1.0 - BETA2) * g.square()
    mean, var = m / (1.0 - BETA1 ** t), v / (1.0 - BETA2 ** t)
    p = st["p"].double() * (1.0 - LR * WD) - LR * mean / (var.sqrt() + ADAM_EPS)
    return p, stored(m, 2, 127.0), stored(v, 4, 255.0), p.clone() if st["copy"] is not None else None
