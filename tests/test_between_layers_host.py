"""Host logic of Dropout, RelativeBias, GroupNorm and the masked attention (no
GPU needed): the operators' calls are replaced by plain torch on the CPU."""
import copy

import pytest
import torch

import approximate_multiplier_dnn_gb300 as am
from approximate_multiplier_dnn_gb300 import layers


@pytest.fixture
def drawn(monkeypatch):
    """Dropout with a mask from (seed, call + step) in plain torch; the calls made."""
    calls = []

    def dropout(x, p, *, seed, call=0, step=None, residual=None):
        number = call + (0 if step is None else int(step))
        calls.append((seed, number))
        g = torch.Generator().manual_seed((seed + 7919 * number) % 2 ** 62)
        y = x * (torch.rand(x.shape, generator=g) >= p) / (1 - p)
        return y if residual is None else y + residual
    monkeypatch.setattr(layers, "dropout", dropout)
    return calls


def test_dropout_layer(drawn):
    layer = layers.Dropout(0.5, generator=torch.Generator().manual_seed(0))
    x, r = torch.ones(1000, requires_grad=True), torch.zeros(1000, requires_grad=True)
    y = layer(x, r)
    y.sum().backward()
    assert torch.equal(x.grad, y.detach()) and torch.equal(r.grad, torch.ones(1000))   # the same mask, drawn again
    assert drawn[0] == drawn[1] and not torch.equal(layer(x), y)                       # another call, another mask
    assert torch.equal(layer(x, r, call=0), y)                                         # a call's mask again
    layer.eval()
    before = len(drawn)
    assert layer(x) is x and torch.equal(layer(x, r), x) and len(drawn) == before
    with pytest.raises(ValueError):
        layers.Dropout(1.0)
    assert layers.Dropout(0.5).draws.seed != layers.Dropout(0.5).draws.seed


def test_dropout_state_goes_on(drawn):
    """A reloaded layer draws what the saved one would have drawn next."""
    a, b = layers.Dropout(0.5, seed=3), layers.Dropout(0.5, seed=4)
    x = torch.ones(100)
    a(x), a(x)
    b.load_state_dict(copy.deepcopy(a.state_dict()))
    assert torch.equal(a(x), b(x)) and drawn[-1] == (3, 2)


def test_step_raised_before_backward_is_refused(drawn):
    """The backward pass would draw another mask than the forward pass's."""
    step = torch.zeros(1, dtype=torch.int64)
    layer = layers.Dropout(0.5, seed=1)
    x = torch.ones(10, requires_grad=True)
    y = layer(x, step=step)
    step += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()
    layer(x, step=step).sum().backward()
    assert drawn[-1] == drawn[-2] == (1, 2)                                            # the second call, step 1


def test_second_derivatives_are_refused(drawn):
    x = torch.ones(10, requires_grad=True)
    (dx,) = torch.autograd.grad((layers.Dropout(0.5)(x) ** 2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_attention_without_dropout_keeps_its_state_dict():
    """An attention layer as it was saved before it could draw loads as before."""
    assert not layers.AMAttention(None).state_dict()
    layers.AMAttention(None).load_state_dict({})
    state = layers.AMAttention(None, dropout=0.1, seed=5).state_dict()
    assert list(state) == ["draws._extra_state"]
    bias = layers.RelativeBias(2, device="cpu")
    assert list(bias.state_dict()) == ["table"] and bias.buckets.dtype == torch.int32
    both = torch.nn.ModuleList([layers.AMAttention(None, bias=bias), layers.AMAttention(None, bias=bias)])
    assert len(list(both.parameters())) == 1                                           # one table, shared
    with pytest.raises(ValueError):
        layers.AMAttention(None, dropout=1.0)


@pytest.fixture
def attention(monkeypatch):
    """The contractions as exact products, the softmax as plain torch."""
    def bgemm(tA, tB, A, B, m, n, k, lut, alpha=1.0):
        return alpha * (A.transpose(1, 2) if tA == "T" else A) @ (B.transpose(1, 2) if tB == "T" else B)

    def logits(s, table, buckets, lengths, causal, offset):
        b, h, q, t = s.shape
        first = offset.view(-1, 1, 1) if isinstance(offset, torch.Tensor) else torch.full((b, 1, 1), offset)
        away = torch.arange(t) - (first + torch.arange(q)[:, None])
        if table is not None:
            D = buckets.numel() // 2
            s = s + table[buckets.long()[away.clamp(-D, D) + D]].permute(0, 3, 1, 2)
        hidden = (away > 0) if causal else torch.zeros_like(away, dtype=torch.bool)
        if lengths is not None:
            hidden = hidden | (torch.arange(t) >= lengths[:, None, None])
        return s.masked_fill(hidden[:, None], -float("inf"))

    def fwd(s, *, table=None, buckets=None, lengths=None, causal=False, offset=0, p=0.0, seed=0, call=0, step=None,
            out=None):
        P = torch.softmax(logits(s, table, buckets, lengths, causal, offset), -1)
        return (P if out is None else out.copy_(P)), None

    def bwd(dp, *, probs=None, scores=None, stats=None, table=None, table_grad=True, out=None, buckets=None, **kw):
        ds = probs * (dp - (probs * dp).sum(-1, keepdim=True))
        return out.copy_(ds), None if table is None or not table_grad else torch.full_like(table, 2.0)
    monkeypatch.setattr(layers, "_f32", lambda t: t.contiguous())
    monkeypatch.setattr(layers, "_bgemm", bgemm)
    monkeypatch.setattr(layers, "attention_softmax", fwd)
    monkeypatch.setattr(layers, "attention_softmax_backward", bwd)
    return logits


def test_masked_attention(attention):
    """Cross attention to padded states of another length with NaN behind a
    length: outputs and gradients as plain torch has them, none for the padding."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn((2, 3, n, 8), generator=g) for n in (5, 7, 7))
    lengths = torch.tensor([7, 4], dtype=torch.int32)
    for t in (k, v):
        t[1, :, 4:] = float("nan")
    q, k, v = (t.requires_grad_() for t in (q, k, v))
    out = layers.am_attention(q, k, v, None, lengths=lengths)
    up = torch.randn(out.shape, generator=g)
    out.backward(up)
    K, V = (t.detach().nan_to_num(0.0).requires_grad_() for t in (k, v))
    Q = q.detach().requires_grad_()
    P = torch.softmax(attention(Q @ K.transpose(2, 3) / 8 ** 0.5, None, None, lengths, False, 0), -1)
    want = P @ V
    want.backward(up)
    assert torch.allclose(out, want, atol=1e-6)
    for got, ref in ((q, Q), (k, K), (v, V)):
        assert torch.allclose(got.grad, ref.grad, atol=1e-6)
    assert not k.grad[1, :, 4:].any() and not v.grad[1, :, 4:].any()


def test_masked_attention_refuses_shapes(attention):
    """Lengths of another shape would hide channels in place of keys where a head
    has as many channels as keys; k and v of another shape would be read as if
    they had the first's."""
    q, k = torch.randn(1, 2, 3, 8), torch.randn(1, 2, 8, 8)
    for lengths in (torch.ones(1, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.tensor(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="lengths"):
            layers.am_attention(q, k, k, None, lengths=lengths)
    for other in (torch.randn(1, 2, 4, 16), torch.randn(2, 1, 8, 8), torch.randn(1, 2, 8, 4), torch.randn(2, 8, 8)):
        with pytest.raises(ValueError, match="k and v"):
            layers.am_attention(q, k, other, None, causal=True)
        with pytest.raises(ValueError, match="k and v"):
            layers.am_attention(q, other, k, None, causal=True)


def test_attention_gives_the_table_its_gradient(attention):
    bias = layers.RelativeBias(3, device="cpu")
    layer = layers.AMAttention(None, bias=bias, causal=True)
    q = torch.randn(2, 3, 5, 8, requires_grad=True)
    out = layer(q, q, q)
    out.sum().backward()
    assert bool((bias.table.grad == 2).all()) and q.grad is not None
    bias.table.requires_grad_(False)
    bias.table.grad = None
    layer(q, q, q, offset=torch.tensor([1, 2], dtype=torch.int32)).sum().backward()
    assert bias.table.grad is None
    with pytest.raises(ValueError):
        layers.am_attention(q, q, q, None, table=bias.table)


def test_even_pixels():
    """Slices of channels go in as they are; anything else is copied."""
    x = torch.arange(2 * 3 * 4 * 6.0).view(2, 3, 4, 6)
    for t, same in ((x, True), (x[..., 1:5], True), (x[:, :, :1], True), (x[..., ::2], False), (x[:, :2], False),
                    (x.transpose(1, 2), False), (x[:1, :2], True), (x.expand(2, 3, 4, 6), True),
                    (x[:1].expand(2, 3, 4, 6), False), (x[..., :1].expand(2, 3, 4, 6), False), (x[:0], True)):
        got = layers._even_pixels(t)
        assert torch.equal(got, t) and (got.data_ptr() == t.data_ptr()) == same
        if got.numel():
            on = type("T", (), dict(shape=got.shape, get_device=lambda s: 0, is_contiguous=lambda s: got.is_contiguous(),
                                    stride=lambda s: got.stride(), is_cuda=True))()
            assert am._pixels("x", on, 0) >= got.shape[-1]


def test_group_norm_layer(monkeypatch):
    calls = []

    def fwd(x, groups, w, b, *, eps, activation, y_dtype):
        calls.append((groups, eps, activation, y_dtype))
        return x * 2, torch.zeros(x.shape[0], groups), torch.ones(x.shape[0], groups)
    monkeypatch.setattr(layers, "group_norm", fwd)
    monkeypatch.setattr(layers, "group_norm_backward",
                        lambda dy, x, w, b, m, r, *, activation: (dy * 2, torch.ones_like(w), torch.zeros_like(b)))
    layer = layers.GroupNorm(2, 8, activation="silu", eps=1e-3, device="cpu")
    x = torch.ones(2, 3, 3, 8, requires_grad=True)
    layer(x).sum().backward()
    assert calls == [(2, 1e-3, "silu", None)] and bool((x.grad == 2).all()) and bool((layer.weight.grad == 1).all())
    with pytest.raises(ValueError):
        layers.GroupNorm(3, 8)
    assert not list(layers.GroupNorm(2, 8, affine=False).parameters())
