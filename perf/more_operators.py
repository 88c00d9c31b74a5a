"""Exact operators between two simulated contractions, as measured cases.

Three operators stand between the contractions of attention and convolution
layers:

softmax  attention's softmax with a learned relative position bias by buckets,
         key lengths (cross attention to a padded encoder), a causal mask and
         dropout of the probabilities; its gradient with the bias table's;
dropout  dropout of a tensor, the mask from a counter-based generator and
         never stored, with an optional residual;
gnorm    group norm with an activation, channels last, and its gradients.

With ``own`` false a case runs in its plain form, elementary torch operations
in fp32 rounded once at the end; with ``own`` true it calls the package.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-5
BUCKETS, DISTANCE = 32, 128      # of the relative position bias
LOW = 0xFFFFFFFF


# ------------------------------------------------------------------ cases
def listed():
    return [
        # training: the framework's attention workload, 16 heads of 512 tokens, both directions
        _softmax("softmax_fwd_batch", "fwd", 32, 16, 512, 512, bias="both", drop=0.1),
        # a decoder's cross attention to encoder states of other, padded lengths; no size is round
        _softmax("softmax_fwd_cross_odd", "fwd", 7, 12, 333, 1531, lengths=True),
        # one generated token against a long cache of two sequences
        _softmax("softmax_fwd_token", "fwd", 2, 16, 1, 131072, bias="past", lengths=True),
        # the first case's backward pass, with the table's gradient; the mask is drawn again
        _softmax("softmax_bwd_batch", "bwd", 32, 16, 512, 512, bias="both", drop=0.1),
        # a causal language model's backward pass at an odd length, no dropout
        _softmax("softmax_bwd_causal_odd", "bwd", 3, 8, 1023, 1023, bias="past", causal=True),
        # the hidden states of four tokens: latency alone
        _dropout("dropout_few", 4096, "f32", False, 0.1),
        # a block's output over an odd number of tokens
        _dropout("dropout_odd", 12_345_677, "f32", False, 0.25),
        # a training batch of 16384 x 4096, added to the residual stream
        _dropout("dropout_batch", 67_108_864, "bf16", True, 0.1),
        # a few small feature maps: latency alone
        _gnorm("gnorm_fwd_few", "fwd", 3, 17, 19, 96, 8, "f32", "silu"),
        # between the 3x3 convolutions of the framework's workload
        _gnorm("gnorm_fwd_batch", "fwd", 128, 32, 32, 64, 8, "f32", "relu"),
        # large feature maps in bf16
        _gnorm("gnorm_fwd_large", "fwd", 8, 128, 128, 512, 32, "bf16", "silu"),
        # training behind the framework's 1x1 convolution
        _gnorm("gnorm_bwd_batch", "bwd", 64, 56, 56, 256, 32, "f32", "silu"),
    ]


def _softmax(name, way, batch, heads, queries, keys, bias="", lengths=False, causal=False, drop=0.0):
    return {"name": name, "op": "softmax", "way": way, "batch": batch, "heads": heads, "queries": queries,
            "keys": keys, "bias": bias, "lengths": lengths, "causal": causal, "drop": drop}


def _dropout(name, n, x, residual, drop):
    return {"name": name, "op": "dropout", "n": n, "x": x, "residual": residual, "drop": drop}


def _gnorm(name, way, batch, height, width, channels, groups, x, act):
    return {"name": name, "op": "gnorm", "way": way, "batch": batch, "height": height, "width": width,
            "channels": channels, "groups": groups, "x": x, "act": act}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("softmax", "softmax", "dropout", "gnorm", "gnorm"))
    most = 1 << 27                               # elements of the largest softmax
    if op == "softmax":
        batch, heads = _log(rng, 1, 32), _log(rng, 1, 16)
        kind = rng.choice(("self", "causal", "cross", "token"))
        if kind == "token":
            queries, keys = 1, _log(rng, 1, min(262144, most // (batch * heads)))
        else:
            side = int(math.sqrt(most // (batch * heads)))
            keys = _log(rng, 8, min(4096, side))
            queries = keys if kind != "cross" else _log(rng, 1, min(2048, side))
            if rng.random() < 0.5:               # padded to a multiple of 8, or as they come
                keys = -(-keys // 8) * 8
                queries = keys if kind != "cross" else queries
        bias = rng.choice(("", "both")) if kind == "self" else "" if kind == "cross" else rng.choice(("", "past"))
        way = "fwd" if kind == "token" else rng.choice(("fwd", "bwd"))
        c = _softmax("", way, batch, heads, queries, keys, bias, kind in ("cross", "token"), kind == "causal",
                     0.0 if kind == "token" else rng.choice((0.0, 0.1)))
    elif op == "dropout":
        c = _dropout("", _log(rng, 1000, 67_108_864), rng.choice(("f32", "bf16")), rng.random() < 0.5,
                     rng.choice((0.05, 0.1, 0.25, 0.5)))
    else:
        groups, each = rng.choice((1, 2, 4, 8, 16, 32)), _log(rng, 1, 48)
        height, batch = _log(rng, 1, 128), _log(rng, 1, 64)
        width = max(1, height + rng.randint(-3, 3))
        batch = max(1, min(batch, (1 << 25) // (height * width * groups * each)))
        c = _gnorm("", rng.choice(("fwd", "bwd")), batch, height, width, groups * each, groups,
                   rng.choice(("f32", "bf16")), rng.choice(("none", "relu", "silu")))
    del c["name"]
    return c


def _lengths(case):
    """Encoder lengths of a padded batch: the first is full, the others down to a third."""
    keys, batch = case["keys"], case["batch"]
    if not case["lengths"]:
        return [keys] * batch
    return [max(1, keys - (2 * keys * b) // (3 * batch)) for b in range(batch)]


def _offset(case, b):
    """Position of a sequence's first query: its last token for a single one."""
    return _lengths(case)[b] - 1 if case["queries"] == 1 else 0


def work(case):
    if case["op"] == "softmax":
        rows = case["batch"] * case["heads"] * case["queries"]
        seen = 0
        for b, n in enumerate(_lengths(case)):
            if case["causal"]:
                first = _offset(case, b) + 1
                full = max(0, min(case["queries"], n - first + 1))     # rows that see fewer than n keys, and n
                seen += full * first + full * (full - 1) // 2 + (case["queries"] - full) * n
            else:
                seen += case["queries"] * n
        seen, out = seen * case["heads"], rows * case["keys"]
        table = 4 * BUCKETS * case["heads"] if case["bias"] else 0
        if case["way"] == "fwd":
            return {"bytes": 4 * (seen + out) + 8 * rows + table, "flops": 5 * seen}
        stats = 8 * rows if case["drop"] else 0
        return {"bytes": 4 * (2 * seen + out) + stats + 2 * table, "flops": 8 * seen}
    if case["op"] == "dropout":
        return {"bytes": case["n"] * SIZE[case["x"]] * (3 if case["residual"] else 2), "flops": 2 * case["n"]}
    e = case["batch"] * case["height"] * case["width"] * case["channels"]
    v = 4 * case["channels"] + 8 * case["batch"] * case["groups"]
    if case["way"] == "fwd":
        return {"bytes": 2 * e * SIZE[case["x"]] + 2 * v, "flops": 8 * e}
    return {"bytes": 3 * e * SIZE[case["x"]] + 4 * v, "flops": 20 * e}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _bucket(distance, both):
    """The bucket of key position minus query position.  With both directions the first half of the buckets is for keys
    up to the query's place and the second for later ones; half of a direction's buckets hold one distance each, the
    rest grow by a constant factor up to DISTANCE, at and beyond which all fall into the last.  In whole numbers, so
    that no distance at a bucket's edge falls to the wrong side."""
    count, first = (BUCKETS // 2, BUCKETS // 2 if distance > 0 else 0) if both else (BUCKETS, 0)
    far = abs(distance) if both else max(0, -distance)
    near = count // 2
    if far < near:
        return first + far
    steps, k = count - near, 0
    # the largest k with near (DISTANCE / near)^(k / steps) <= far
    while k + 1 < steps and DISTANCE ** (k + 1) * near ** steps <= far ** steps * near ** (k + 1):
        k += 1
    return first + near + k


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case), "seed": 1_000_003 * (seed + 1), "call": 3}
    if case["op"] == "softmax":
        B, H, Q, K = case["batch"], case["heads"], case["queries"], case["keys"]
        st["scores"] = _randn(g, B, H, Q, K).mul_(1.5)
        st["table"] = _randn(g, BUCKETS, H) if case["bias"] else None
        st["map"] = None
        if case["bias"]:                         # kept by the layer, one entry for each distance
            st["map"] = torch.tensor([_bucket(d, case["bias"] == "both") for d in range(-DISTANCE, DISTANCE + 1)],
                                     dtype=torch.int32, device="cuda")
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["lengths"] else None
        st["offset"] = 0
        if Q == 1:
            st["offset"] = torch.tensor([_offset(case, b) for b in range(B)], dtype=torch.int32, device="cuda")
        if case["way"] == "bwd":                 # what the forward pass left, and the gradient
            st["dprobs"] = _randn(g, B, H, Q, K).mul_(0.1)
            probs, st["stats"] = _softmax_fwd_plain(st)
            if not case["drop"]:                 # the probabilities are enough, the scores are gone
                st["probs"] = probs
                del st["scores"]
    elif case["op"] == "dropout":
        st["x"] = _randn(g, case["n"]).to(TYPES[case["x"]])
        st["residual"] = _randn(g, case["n"]).to(TYPES[case["x"]]) if case["residual"] else None
    else:
        shape, C, G = (case["batch"], case["height"], case["width"], case["channels"]), case["channels"], case["groups"]
        X = TYPES[case["x"]]
        st["x"] = (_randn(g, *shape) * (0.5 + torch.rand(C, generator=g, device="cuda")) + 0.3 * _randn(g, C)).to(X)
        st["w"], st["b"] = 1.0 + 0.1 * _randn(g, C), 0.1 * _randn(g, C)
        if case["way"] == "bwd":
            st["dy"] = (0.01 * _randn(g, *shape)).to(X)
            _, st["mean"], st["rstd"] = _gnorm_fwd_plain(st)
    return st


# ------------------------------------------------------------------ plain forms
def _words(quads, call, seed):
    """The four 32-bit words of each quad's number under Philox4x32-10, as int64."""
    c0, c1 = quads & LOW, quads >> 32
    c2, c3 = torch.full_like(quads, call & LOW), torch.full_like(quads, call >> 32)
    k0, k1 = seed & LOW, (seed >> 32) & LOW
    for _ in range(10):
        # a product's low 64 bits are right in int64 also where it wraps
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & LOW) ^ c1 ^ k0, b & LOW, ((a >> 32) & LOW) ^ c3 ^ k1, a & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return torch.stack((c0, c1, c2, c3), -1)


def _kept(rows, cols, st):
    """Which elements of a matrix of rows x cols stay: a quad of numbers for every four of a row."""
    quads = -(-cols // 4)
    out, step = torch.empty((rows, cols), dtype=torch.bool, device="cuda"), max(1, (1 << 24) // quads)
    border = round(st["case"]["drop"] * 2 ** 32)
    for a in range(0, rows, step):               # some rows at a time: the words are eight bytes each
        n = min(step, rows - a)
        if rows == 1:                            # one long row, in pieces of its quads
            for q in range(0, quads, 1 << 22):
                w = _words(torch.arange(q, min(quads, q + (1 << 22)), device="cuda"), st["call"], st["seed"])
                out[0, 4 * q:4 * q + w.numel()] = (w >= border).view(-1)[:cols - 4 * q]
            break
        w = _words(torch.arange(a * quads, (a + n) * quads, device="cuda"), st["call"], st["seed"])
        out[a:a + n] = (w >= border).view(n, 4 * quads)[:, :cols]
    return out


def _positions(st):
    """[batch or 1, 1, queries, 1] positions of the queries, and the keys' [keys]."""
    c = st["case"]
    i, j = torch.arange(c["queries"], device="cuda"), torch.arange(c["keys"], device="cuda")
    first = st["offset"].long().view(-1, 1, 1, 1) if torch.is_tensor(st["offset"]) else st["offset"]
    return (first + i.view(1, 1, -1, 1)), j


def _visible(st):
    c = st["case"]
    pos, j = _positions(st)
    see = torch.ones((1, 1, 1, c["keys"]), dtype=torch.bool, device="cuda")
    if st["lengths"] is not None:
        see = see & (j < st["lengths"].view(-1, 1, 1, 1))
    return see & (j <= pos) if c["causal"] else see


def _row_buckets(st):
    pos, j = _positions(st)
    return st["map"].long()[(j - pos).clamp(-DISTANCE, DISTANCE) + DISTANCE]     # [batch or 1, 1, queries, keys]


def _softmax_fwd_plain(st):
    c = st["case"]
    a = st["scores"]
    if c["bias"]:
        a = a + st["table"][_row_buckets(st)[:, 0]].permute(0, 3, 1, 2)
    a = a.masked_fill(~_visible(st), -math.inf)
    top = a.amax(-1, keepdim=True)
    e = (a - top).exp()
    inv = 1.0 / e.sum(-1, keepdim=True)
    p = e * inv
    stats = torch.cat((top, inv), -1)
    if c["drop"]:
        keep = _kept(p[..., 0].numel(), c["keys"], st).view(p.shape)
        p = torch.where(keep, p * (1.0 / (1.0 - c["drop"])), torch.zeros_like(p))
    return p, stats


def _softmax_bwd_plain(st):
    c = st["case"]
    g = st["dprobs"]
    if c["drop"]:
        a = st["scores"]
        if c["bias"]:
            a = a + st["table"][_row_buckets(st)[:, 0]].permute(0, 3, 1, 2)
        p = ((a - st["stats"][..., :1]).exp() * st["stats"][..., 1:]).masked_fill(~_visible(st), 0.0)
        keep = _kept(p[..., 0].numel(), c["keys"], st).view(p.shape)
        g = torch.where(keep, g * (1.0 / (1.0 - c["drop"])), torch.zeros_like(g))
    else:
        p = st["probs"]
    ds = p * (g - (p * g).sum(-1, keepdim=True))
    if not c["bias"]:
        return ds, None
    per = ds.sum(0)                              # every sequence starts at the same place: [heads, queries, keys]
    which, table = _row_buckets(st)[0, 0], torch.empty_like(st["table"])
    for k in range(BUCKETS):
        table[k] = (per * (which == k)).sum((1, 2))
    return ds, table


def _dropout_plain(st):
    x = st["x"].float()
    y = torch.where(_kept(1, x.numel(), st)[0], x * (1.0 / (1.0 - st["case"]["drop"])), torch.zeros_like(x))
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(st["x"].dtype)


def _grouped(t, groups):
    """[batch, pixels, groups, channels of a group]"""
    return t.reshape(t.shape[0], -1, groups, t.shape[-1] // groups)


def _gnorm_fwd_plain(st):
    c = st["case"]
    x = _grouped(st["x"].float(), c["groups"])
    mean = x.mean((1, 3), keepdim=True)
    rstd = 1.0 / ((x - mean).square().mean((1, 3), keepdim=True) + EPS).sqrt()
    z = ((x - mean) * rstd).reshape(st["x"].shape) * st["w"] + st["b"]
    if c["act"] == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif c["act"] == "silu":
        z = z * (1.0 / (1.0 + (-z).exp()))
    return z.to(st["x"].dtype), mean[:, 0, :, 0].contiguous(), rstd[:, 0, :, 0].contiguous()


def _gnorm_bwd_plain(st):
    c = st["case"]
    G = c["groups"]
    mean, rstd = st["mean"][:, None, :, None], st["rstd"][:, None, :, None]
    xh = ((_grouped(st["x"].float(), G) - mean) * rstd).reshape(st["x"].shape)
    dz = st["dy"].float()
    if c["act"] == "relu":                       # the sign of z in 64 bits: it decides the whole gradient
        x64 = (_grouped(st["x"].double(), G) - mean) * rstd
        dz = dz * (x64.reshape(xh.shape) * st["w"] + st["b"] > 0)
        del x64
    elif c["act"] == "silu":
        z = xh * st["w"] + st["b"]
        s = 1.0 / (1.0 + (-z).exp())
        dz = dz * (s * (1.0 + z * (1.0 - s)))
    dw, db = (dz * xh).sum((0, 1, 2)), dz.sum((0, 1, 2))
    t, h = _grouped(dz * st["w"], G), _grouped(xh, G)
    dx = rstd * (t - t.mean((1, 3), keepdim=True) - h * (t * h).mean((1, 3), keepdim=True))
    return dx.reshape(st["x"].shape).to(st["x"].dtype), dw, db


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    fwd = c.get("way") == "fwd"
    if not own:
        if c["op"] == "dropout":
            return _dropout_plain(st)
        if c["op"] == "softmax":
            return _softmax_fwd_plain(st) if fwd else _softmax_bwd_plain(st)
        return _gnorm_fwd_plain(st) if fwd else _gnorm_bwd_plain(st)
    import approximate_multiplier_dnn_gb300 as am
    if c["op"] == "dropout":
        return am.dropout(st["x"], c["drop"], seed=st["seed"], call=st["call"], residual=st["residual"])
    if c["op"] == "softmax":
        kw = dict(table=st["table"], buckets=st["map"], lengths=st["lengths"], causal=c["causal"],
                  offset=st["offset"], p=c["drop"], seed=st["seed"], call=st["call"])
        if fwd:
            return am.attention_softmax(st["scores"], **kw)
        if c["drop"]:
            return am.attention_softmax_backward(st["dprobs"], scores=st["scores"], stats=st["stats"], **kw)
        return am.attention_softmax_backward(st["dprobs"], probs=st["probs"], **kw)
    if fwd:
        return am.group_norm(st["x"], c["groups"], st["w"], st["b"], eps=EPS, activation=c["act"])
    return am.group_norm_backward(st["dy"], st["x"], st["w"], st["b"], st["mean"], st["rstd"], activation=c["act"])


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "dropout":
        keep = _stays(torch.arange(case["n"], device="cuda"), st)
        y = st["x"].double() * keep / (1.0 - case["drop"])
        return y if st["residual"] is None else y + st["residual"].double()
    if case["op"] == "softmax":
        return _softmax_exact(st)
    return _gnorm_fwd_exact(st) if case["way"] == "fwd" else _gnorm_bwd_exact(st)


def _stays(index, st):
    """Which of the elements with these numbers stay: Philox4x32-10 of element // 4, products by halves of 16 bits."""
    out = torch.empty(index.shape, dtype=torch.bool, device=index.device)
    flat, seen, border = index.reshape(-1), out.view(-1), int(2 ** 32 * st["case"]["drop"] + 0.5)
    for a in range(0, flat.numel(), 1 << 25):
        n = flat[a:a + (1 << 25)]
        q, word = torch.div(n, 4, rounding_mode="floor"), n % 4
        ctr = [q % 2 ** 32, torch.div(q, 2 ** 32, rounding_mode="floor"), q * 0 + st["call"] % 2 ** 32,
               q * 0 + st["call"] // 2 ** 32]
        for r in range(10):
            key = [(st["seed"] + r * 0x9E3779B9) % 2 ** 32, (st["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
            hi0, lo0 = _product(ctr[0], 0xD2511F53)
            hi1, lo1 = _product(ctr[2], 0xCD9E8D57)
            ctr = [hi1 ^ ctr[1] ^ key[0], lo1, hi0 ^ ctr[3] ^ key[1], lo0]
        number = torch.where(word < 2, torch.where(word == 0, ctr[0], ctr[1]), torch.where(word == 2, ctr[2], ctr[3]))
        seen[a:a + n.numel()] = number >= border
    return out


def _product(x, m):
    """High and low 32 bits of x m by schoolbook halves; no part exceeds 2^33."""
    xl, xh, ml, mh = x % 65536, x // 65536, m % 65536, m // 65536
    low, mid1, mid2 = xl * ml, xl * mh, xh * ml
    middle = low // 65536 + mid1 % 65536 + mid2 % 65536
    return xh * mh + mid1 // 65536 + mid2 // 65536 + middle // 65536, low % 65536 + (middle % 65536) * 65536


def _softmax_exact(st):
    """Head by head from the definition; the bias is looked up distance by distance."""
    c = st["case"]
    B, H, Q, K = c["batch"], c["heads"], c["queries"], c["keys"]
    fwd = c["way"] == "fwd"
    out = torch.zeros((B, H, Q, K), dtype=torch.float64, device="cuda")
    stats = torch.zeros((B, H, Q, 2), dtype=torch.float64, device="cuda")
    dtable = torch.zeros((BUCKETS, H), dtype=torch.float64, device="cuda") if c["bias"] else None
    i, j = torch.arange(Q, device="cuda")[:, None], torch.arange(K, device="cuda")[None]
    lengths = _lengths(c)
    for b in range(B):
        away = j - i - _offset(c, b)
        near = torch.minimum(torch.maximum(away, away * 0 - DISTANCE), away * 0 + DISTANCE)
        hidden = (j >= lengths[b]) | ((away > 0) if c["causal"] else torch.zeros_like(away, dtype=torch.bool))
        for h in range(H):
            row = (b * H + h) * Q + i
            stays = _stays(row * (4 * ((K + 3) // 4)) + j, st) if c["drop"] else None
            if fwd or c["drop"]:
                z = st["scores"][b, h].double()
                if c["bias"]:
                    of_distance = st["table"][:, h].double()[st["map"].long()]
                    z = z + of_distance[near + DISTANCE]
                z = torch.where(hidden, -math.inf, z)
            if fwd:
                p = torch.softmax(z, 1)
                stats[b, h, :, 0] = z.max(1).values
                stats[b, h, :, 1] = torch.exp(stats[b, h, :, 0] - torch.logsumexp(z, 1))
                out[b, h] = p * stays / (1.0 - c["drop"]) if c["drop"] else p
                continue
            up = st["dprobs"][b, h].double()
            if c["drop"]:                        # the statistics are inputs, as the forward pass left them
                p = torch.exp(z - st["stats"][b, h, :, :1].double()) * st["stats"][b, h, :, 1:].double()
                up = up * stays / (1.0 - c["drop"])
            else:
                p = st["probs"][b, h].double()
            ds = p * up - p * torch.einsum("qk,qk->q", p, up)[:, None]
            out[b, h] = ds
            if c["bias"]:
                dtable[:, h].index_add_(0, st["map"].long(), torch.zeros(2 * DISTANCE + 1, dtype=torch.float64,
                                        device="cuda").index_add_(0, (near + DISTANCE).reshape(-1), ds.reshape(-1)))
    return (out, stats) if fwd else (out, dtable)


def _act_exact(z, act):
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    s = torch.sigmoid(z)
    return z * s, s + z * s * (1 - s)


def _gnorm_fwd_exact(st):
    c = st["case"]
    G = c["groups"]
    y = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda")
    mean, rstd = (torch.empty((c["batch"], G), dtype=torch.float64, device="cuda") for _ in range(2))
    size = c["channels"] // G
    for n in range(c["batch"]):
        for g in range(G):
            s = slice(g * size, (g + 1) * size)
            x = st["x"][n, ..., s].double()
            var, m = torch.var_mean(x, correction=0)
            mean[n, g], rstd[n, g] = m, (var + EPS).pow(-0.5)
            y[n, ..., s] = _act_exact((x - m) * rstd[n, g] * st["w"][s].double() + st["b"][s].double(), c["act"])[0]
    return y, mean, rstd


def _gnorm_bwd_exact(st):
    """By the chain rule from x - mean and rstd, the forward's statistics as they are."""
    c = st["case"]
    G, size = c["groups"], c["channels"] // c["groups"]
    dx = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda")
    dw, db = (torch.zeros(c["channels"], dtype=torch.float64, device="cuda") for _ in range(2))
    m = size * c["height"] * c["width"]
    for n in range(c["batch"]):
        for g in range(G):
            s = slice(g * size, (g + 1) * size)
            r, w = st["rstd"][n, g].double(), st["w"][s].double()
            d = st["x"][n, ..., s].double() - st["mean"][n, g].double()
            up = st["dy"][n, ..., s].double() * _act_exact(d * r * w + st["b"][s].double(), c["act"])[1]
            dw[s] += (up * d * r).sum((0, 1))
            db[s] += up.sum((0, 1))
            up = up * w
            # rstd = (mean d^2 + eps)^(-1/2): d(rstd)/d(d) = -rstd^3 d / m
            centre = up * r - d * ((up * d).sum() * r.pow(3) / m)
            dx[n, ..., s] = centre - (up * r).sum() / m
    return dx, dw, db
