"""The AdamW step.  The ABI fixes each fp32 operation and its order, so numpy's
fp32 (correctly rounded, no contraction) gives the same bits; against the
formula in 64 bits the new moments are within 3 roundings of their terms, and
the parameter within 3 roundings of itself and 12 of its update."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B1, B2, EPS, LR, WD = 0.9, 0.999, 1e-8, 3e-4, 0.1
BLOCK = 256
f32 = np.float32


def decode(q, scale, second):
    t = q.astype(f32) * f32(1.0 / (255.0 if second else 127.0))
    t2 = t * np.abs(t)
    return (t2 * t2 if second else t2) * np.repeat(scale, BLOCK)[:q.size]


def encode(x, second):
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK, f32)
    pad[:n] = x
    b = pad.reshape(-1, BLOCK)
    scale = np.abs(b).max(1)
    top = f32(255.0 if second else 127.0)
    root = np.sqrt(np.sqrt(scale)) if second else np.sqrt(scale)
    k = np.divide(top, root, out=np.zeros_like(root), where=root > 0)
    f = np.sqrt(np.sqrt(b)) if second else np.sqrt(np.abs(b))
    q = np.minimum(np.rint(f * k[:, None]), top)
    q = np.where(b > 0, np.maximum(q, 1), q) if second else np.where(b < 0, -q, q)
    return q.astype(np.uint8 if second else np.int8).reshape(-1)[:n], scale


def adam32(p, g, m, v, step, gs=None, lr=LR, wd=WD):
    """The documented operations, each rounded to fp32."""
    g = g.astype(f32) if gs is None else g.astype(f32) * f32(gs)
    m = m * f32(B1) + g * f32(1.0 - B1)
    v = v * f32(B2) + (g * g) * f32(1.0 - B2)
    u = m / (np.sqrt(v) * f32(1.0 / np.sqrt(1.0 - B2 ** step)) + f32(EPS))
    return p * f32(1.0 - lr * wd) - u * f32(lr / (1.0 - B1 ** step)), m, v


def inputs(n, seed, g_bf16=False):
    import torch
    g = torch.Generator().manual_seed(seed)
    p = torch.randn(n, generator=g) * 0.02
    grad = torch.randn(n, generator=g) * 1e-3
    m = torch.randn(n, generator=g) * 3e-4
    v = torch.randn(n, generator=g).square() * 1e-6
    return p, grad.to(torch.bfloat16) if g_bf16 else grad, m, v


SIZES = [1, 7, 8, 255, 256, 257, 4095, 4096, 4097, 20_001]


@pytest.mark.parametrize("g_bf16", [False, True])
@pytest.mark.parametrize("off", [0, 1])
def test_fp32_moments(amd, g_bf16, off):
    """Several tensors in one step, aligned or one element off, with copies;
    neighbours of each tensor in its buffer stay as they are."""
    import torch
    table, hold, want = [], [], []
    gs = torch.full((1,), 0.5, device="cuda")
    for i, n in enumerate(SIZES):
        p, g, m, v = inputs(n, i, g_bf16)

        def place(t):
            buf = torch.full((n + off + 8,), 9.0, dtype=t.dtype, device="cuda")
            buf[off:off + n] = t.cuda()
            return buf, buf[off:off + n]
        bufs = [place(t) for t in (p, g, m, v, p.to(torch.bfloat16))]
        table.append(amd.AdamwTensor.make(bufs[0][1], bufs[1][1], bufs[2][1], bufs[3][1],
                                          copy=bufs[4][1] if i % 2 else None, weight_decay=WD))
        hold.append(bufs)
        want.append(adam32(p.numpy(), g.float().numpy(), m.numpy(), v.numpy(), 3, 0.5))
    amd.adamw_step(amd.adamw_table(table), lr=LR, beta1=B1, beta2=B2, eps=EPS, step=3, grad_scale=gs)
    torch.cuda.synchronize()
    for i, (bufs, (p, m, v)) in enumerate(zip(hold, want)):
        for (buf, t), w in zip((bufs[0], bufs[2], bufs[3]), (p, m, v)):
            assert np.array_equal(t.cpu().numpy(), w), SIZES[i]
        if i % 2:
            assert torch.equal(bufs[4][1].cpu(), torch.from_numpy(p).to(torch.bfloat16))
        for buf, t in bufs:
            assert bool((buf[:off] == 9.0).all()) and bool((buf[off + t.numel():] == 9.0).all())


@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 7])
def test_against_64_bits(amd, step):
    import torch
    n = 5000
    p, g, m, v = inputs(n, step)
    d = [t.cuda() for t in (p, g, m, v)]
    amd.adamw_step(amd.adamw_table([amd.AdamwTensor.make(*d, weight_decay=WD, lr_scale=0.5)]), lr=LR, beta1=B1,
                   beta2=B2, eps=EPS, step=step)
    P, G, M, V = (t.double().numpy() for t in (p, g, m, v))
    m64, v64 = B1 * M + (1 - B1) * G, B2 * V + (1 - B2) * G * G
    upd = LR / 2 * (m64 / (1 - B1 ** step)) / (np.sqrt(v64 / (1 - B2 ** step)) + EPS)
    p64 = P * (1 - LR / 2 * WD) - upd
    got = [t.cpu().double().numpy() for t in d]
    m_err = 4 * U * (np.abs(B1 * M) + np.abs((1 - B1) * G))
    assert np.all(np.abs(got[2] - m64) <= m_err)
    assert np.all(np.abs(got[3] - v64) <= 5 * U * v64)
    # the update inherits the first moment's error relative to it
    assert np.all(np.abs(got[0] - p64) <= 3 * U * np.abs(P) + 14 * U * np.abs(upd) +
                  np.abs(upd) * m_err / np.maximum(np.abs(m64), 1e-300) + 1e-40)


def state8(m, v):
    import torch
    mq, ms = encode(m.numpy(), False)
    vq, vs = encode(v.numpy(), True)
    return [torch.from_numpy(t).cuda() for t in (mq, vq, ms, vs)], (mq, vq, ms, vs)


@pytest.mark.parametrize("g_bf16", [False, True])
@pytest.mark.parametrize("off", [0, 3])
def test_8_bit_moments(amd, g_bf16, off):
    """Codes, scales, parameters and read-back values to the bit, at sizes
    with a short last block, aligned or not."""
    import torch
    table, hold = [], []
    for i, n in enumerate(SIZES):
        p, g, m, v = inputs(n, 50 + i, g_bf16)
        if n >= 256:
            m[:256], v[:256], g[:256] = 0.0, 0.0, 0.0          # a block that is all zero
        (mq, vq, ms, vs), host = state8(m, v)

        def place(t):
            buf = torch.zeros(n + off, dtype=t.dtype, device="cuda")
            buf[off:] = t.cuda()
            return buf[off:]
        d = [place(t) for t in (p, g, mq, vq)]
        table.append(amd.AdamwTensor.make(*d, m_scale=ms, v_scale=vs, weight_decay=WD))
        hold.append((d, ms, vs, p, g, host))
    amd.adamw_step(amd.adamw_table(table), lr=LR, beta1=B1, beta2=B2, eps=EPS, step=7)
    for d, ms, vs, p, g, (mq, vq, hms, hvs) in hold:
        want, m, v = adam32(p.numpy(), g.float().numpy(), decode(mq, hms, False), decode(vq, hvs, True), 7)
        wm, wms = encode(m, False)
        wv, wvs = encode(v, True)
        assert np.array_equal(d[0].cpu().numpy(), want)
        assert np.array_equal(d[2].cpu().numpy(), wm) and np.array_equal(d[3].cpu().numpy(), wv)
        assert np.array_equal(ms.cpu().numpy(), wms) and np.array_equal(vs.cpu().numpy(), wvs)
        assert np.array_equal(amd.adamw_moment_values(d[2], ms).cpu().numpy(), decode(wm, wms, False))
        assert np.array_equal(amd.adamw_moment_values(d[3], vs).cpu().numpy(), decode(wv, wvs, True))


@pytest.mark.parametrize("size", [1e-14, 1e-18, 1e-22, 1e15])
def test_8_bit_moments_of_any_size(amd, size):
    """Gradients whose moments are near fp32's ends, a step of the state from zero: the documented bits."""
    import torch
    n = 3000
    p, g, _, _ = inputs(n, 21)
    g = g * float(size) * 1e3
    g[::3] *= 1e-4
    zero = np.zeros(n, f32)
    (mq, vq, ms, vs), host = state8(torch.zeros(n), torch.zeros(n))
    d = p.cuda()
    amd.adamw_step(amd.adamw_table([amd.AdamwTensor.make(d, g.cuda(), mq, vq, m_scale=ms, v_scale=vs)]), lr=LR,
                   beta1=B1, beta2=B2, eps=EPS, step=1)
    want, m, v = adam32(p.numpy(), g.numpy(), zero, zero, 1, wd=0.0)
    wm, wms = encode(m, False)
    wv, wvs = encode(v, True)
    assert np.array_equal(d.cpu().numpy(), want)
    assert np.array_equal(mq.cpu().numpy(), wm) and np.array_equal(ms.cpu().numpy(), wms)
    assert np.array_equal(vq.cpu().numpy(), wv) and np.array_equal(vs.cpu().numpy(), wvs)


def test_8_bit_moments_of_a_large_tensor(amd):
    """Enough elements for blocks of several passes, with a ragged end: every
    tensor moves as it does in a step of its own."""
    import torch
    sizes = [7_000_001, 3_500_130, 255, 4096 * 8 + 17]
    parts = [[t.cuda() for t in inputs(n, 30 + i, True)] for i, n in enumerate(sizes)]
    state = []
    for p, g, m, v in parts:
        nb = -(-p.numel() // BLOCK)
        q = [torch.zeros(p.numel(), dtype=torch.int8, device="cuda"), torch.zeros(p.numel(), dtype=torch.uint8, device="cuda"),
             torch.zeros(nb, device="cuda"), torch.zeros(nb, device="cuda")]
        state.append([p] + q + [torch.zeros(p.numel(), dtype=torch.bfloat16, device="cuda")])
    other = [[t.clone() for t in st] for st in state]

    def entry(st, g):
        return amd.AdamwTensor.make(st[0], g, st[1], st[2], m_scale=st[3], v_scale=st[4], copy=st[5], weight_decay=WD)
    for step in (1, 2):
        amd.adamw_step(amd.adamw_table([entry(st, p[1]) for st, p in zip(state, parts)]), lr=LR, step=step)
        for st, p in zip(other, parts):
            chunk = 4096 * BLOCK                         # whole blocks, few enough for one pass each
            for a in range(0, p[0].numel(), chunk):
                b, s = min(a + chunk, p[0].numel()), a // BLOCK
                e = -(-b // BLOCK)
                cut = [st[0][a:b], st[1][a:b], st[2][a:b], st[3][s:e], st[4][s:e], st[5][a:b]]
                amd.adamw_step(amd.adamw_table([entry(cut, p[1][a:b])]), lr=LR, step=step)
    for st, ot in zip(state, other):
        assert all(torch.equal(x, y) for x, y in zip(st, ot))


def test_8_bit_codes_are_near_their_values(amd):
    """Nearest code in the root domain: the first moment's root is within half
    a step (1/254 of the block's root), the second's fourth root within 1/510,
    a second moment above zero reads back above zero, zero as zero."""
    import torch
    n = 4096
    p, g, m, v = inputs(n, 5)
    v[::7] = 0.0
    g[::7] = 0.0
    v[1::7] *= 1e-12
    g[1::7] *= 1e-6
    (mq, vq, ms, vs), host = state8(m, v)
    m0, v0 = decode(host[0], host[2], False).astype(np.float64), decode(host[1], host[3], True).astype(np.float64)
    G = g.double().numpy()
    amd.adamw_step(amd.adamw_table([amd.AdamwTensor.make(p.cuda(), g.cuda(), mq, vq, m_scale=ms, v_scale=vs)]), lr=LR,
                   beta1=B1, beta2=B2, eps=EPS, step=1)
    m64, v64 = B1 * m0 + (1 - B1) * G, B2 * v0 + (1 - B2) * G * G
    got_m = amd.adamw_moment_values(mq, ms).cpu().double().numpy()
    got_v = amd.adamw_moment_values(vq, vs).cpu().double().numpy()
    top_m = np.repeat(np.abs(m64).reshape(-1, BLOCK).max(1), BLOCK)
    top_v = np.repeat(v64.reshape(-1, BLOCK).max(1), BLOCK)
    slack = 1e-5
    root = np.sqrt(np.abs(got_m) / top_m) * np.sign(got_m) - np.sqrt(np.abs(m64) / top_m) * np.sign(m64)
    assert np.abs(root).max() <= 1 / 254 + slack
    r4 = (got_v / top_v) ** 0.25 - (v64 / top_v) ** 0.25
    tiny = (v64 / top_v) ** 0.25 < 0.5 / 255                   # rounds up to code 1
    assert np.abs(r4[~tiny]).max() <= 1 / 510 + slack and np.abs(r4[tiny]).max() <= 1 / 255 + slack
    assert np.all((got_v > 0) == (v64 > 0)) and not got_v[::7].any()


def test_non_finite_gradient_marks_its_block(amd):
    import torch
    p, g, m, v = inputs(1024, 8)
    g[300] = float("nan")
    g[700] = float("inf")
    (mq, vq, ms, vs), _ = state8(m, v)
    d = p.cuda()
    amd.adamw_step(amd.adamw_table([amd.AdamwTensor.make(d, g.cuda(), mq, vq, m_scale=ms, v_scale=vs)]), lr=LR, step=1)
    bad = torch.tensor([False, True, True, False])
    for q, s in ((mq, ms), (vq, vs)):
        assert torch.equal(torch.isnan(s.cpu()), bad)
        assert torch.equal(torch.isnan(amd.adamw_moment_values(q, s).cpu()).view(4, 256).all(1), bad)
    assert torch.equal(torch.isfinite(d.cpu()).logical_not().nonzero()[:, 0], torch.tensor([300, 700]))


@pytest.mark.parametrize("count", [9, 65, 900])
def test_many_tensors(amd, count):
    """Each size of a launch's tensor list, and more tensors than one launch takes."""
    import torch
    n = [(i * 37) % 900 for i in range(count)]                 # some empty
    flat = [t.cuda() for t in inputs(sum(n) + 1, 1)]
    one = [t.clone() for t in flat]
    at = np.concatenate([[0], np.cumsum(n)])
    table = [amd.AdamwTensor.make(*(t[a:b] for t in flat), weight_decay=WD) for a, b in zip(at, at[1:])]
    before = amd.amsim_kernel_launches()
    amd.adamw_step(amd.adamw_table(table), lr=LR, step=4)
    assert amd.amsim_kernel_launches() - before == -(-sum(1 for x in n if x) // 400)
    end = int(at[-1])
    amd.adamw_step(amd.adamw_table([amd.AdamwTensor.make(*(t[:end] for t in one), weight_decay=WD)]), lr=LR, step=4)
    for a, b in zip(flat, one):
        assert torch.equal(a, b)


def test_graph_replay(amd):
    import torch
    a = [t.cuda() for t in inputs(3000, 2)]
    b = [t.clone() for t in a]
    gs = torch.ones(1, device="cuda")
    table = amd.adamw_table([amd.AdamwTensor.make(*a)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        amd.adamw_step(table, lr=LR, step=1, grad_scale=gs)
    for scale in (1.0, 0.25):
        gs.fill_(scale)
        graph.replay()
        amd.adamw_step(amd.adamw_table([amd.AdamwTensor.make(*b)]), lr=LR, step=1,
                       grad_scale=torch.full((1,), scale, device="cuda"))
    for p, q in zip(a, b):
        assert torch.equal(p, q)


@pytest.mark.parametrize("eight", [False, True])
def test_offsets_past_32_bits(amd, eight):
    """A tensor of more than 2^31 elements: its end moves as a small tensor does."""
    import torch
    n, tail = 2 ** 31 + 5000, 4000
    p, g, m, v = inputs(tail, 3, True)
    big = dict(device="cuda")
    start = n - tail
    assert start % BLOCK == 1000 % BLOCK
    P = torch.zeros(n, **big)
    G = torch.zeros(n, dtype=torch.bfloat16, **big)
    P[start:], G[start:] = p.cuda(), g.cuda()
    kw = {}
    if eight:
        M, V = torch.zeros(n, dtype=torch.int8, **big), torch.zeros(n, dtype=torch.uint8, **big)
        blocks = -(-n // BLOCK)
        kw = dict(m_scale=torch.zeros(blocks, **big), v_scale=torch.zeros(blocks, **big))
    else:
        M, V = torch.zeros(n, **big), torch.zeros(n, **big)
    amd.adamw_step(amd.adamw_table([amd.AdamwTensor.make(P, G, M, V, **kw)]), lr=LR, beta1=B1, beta2=B2, eps=EPS,
                   step=1)
    zero = np.zeros(tail, f32)
    want, wm, wv = adam32(p.numpy(), g.float().numpy(), zero, zero, 1, wd=0.0)
    assert np.array_equal(P[start:].cpu().numpy(), want)
    assert not P[:1000].any() and not P[start - 5000:start].any()
    if eight:
        lead = start % BLOCK                       # elements of the tail's first block before it
        pad = np.concatenate([np.zeros(lead, f32), wm])
        q, s = encode(pad, False)
        assert np.array_equal(M[start:].cpu().numpy(), q[lead:])
        assert np.array_equal(kw["m_scale"][start // BLOCK:].cpu().numpy(), s)
    else:
        assert np.array_equal(M[start:].cpu().numpy(), wm) and np.array_equal(V[start:].cpu().numpy(), wv)
