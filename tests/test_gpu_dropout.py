"""Dropout against its definition: the generator in plain integers, one fp32
product, an addition and one rounding."""
import numpy as np
import pytest

from philox_reference import stays

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(n, dtype, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, generator=g, device="cuda").to(getattr(torch, dtype))


def want(x, residual, p, call, seed):
    """In 64 bits, and the magnitude of the product."""
    x = x.double().cpu().numpy().reshape(-1)
    keep = stays(1, x.size, p, call, seed)[0]
    prod = np.where(keep, x / (1 - p), 0.0)
    return prod + (0 if residual is None else residual.double().cpu().numpy().reshape(-1)), np.abs(prod), keep


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 1023, 4096, 16384, 16387, 100_003])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(amd, n, dtype, residual):
    """The factor and the product are each off by at most U, the sum and a
    bf16 result by half a step."""
    x, r = make(n, dtype, 1), make(n, dtype, 2) if residual else None
    for p, seed, call in ((0.1, 12345, 0), (0.5, -7, 2 ** 40 + 3), (0.9, 2 ** 63 + 11, 2 ** 63)):
        y = amd.dropout(x, p, seed=seed, call=call, residual=r)
        ref, prod, keep = want(x, r, p, call, seed)
        got = y.double().cpu().numpy()
        assert y.dtype == x.dtype and y.shape == x.shape
        half = U if dtype == "float32" else 2.0 ** -8
        assert np.all(np.abs(got - ref) <= 3 * U * prod + half * (np.abs(ref) + 3 * U * prod))
        if r is None:
            assert np.array_equal(got != 0, keep & (x.double().cpu().numpy() != 0))


@pytest.mark.parametrize("off", range(8))
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_any_alignment(amd, off, dtype):
    """Tensors off 16 bytes: the same values bit for bit, and nothing beside them."""
    import torch
    n = 5003
    x, r = make(n, dtype, 3), make(n, dtype, 4)
    ref = amd.dropout(x, 0.3, seed=5, residual=r)
    places = []
    for t in (x, r, torch.zeros_like(x)):
        buf = torch.full((n + 32,), 7.0, dtype=x.dtype, device="cuda")
        buf[off:off + n] = t
        places.append(buf)
    d = amd.DropoutDesc(0.3, 5, 0, None)
    a, b, c = (buf[off:off + n] for buf in places)
    amd.amsim_dropout(d, amd.AMSIM_F32 if dtype == "float32" else amd.AMSIM_BF16, n, a, b, c)
    assert torch.equal(c, ref)
    assert bool((places[2][:off] == 7).all()) and bool((places[2][off + n:] == 7).all())
    amd.amsim_dropout(d, amd.AMSIM_F32 if dtype == "float32" else amd.AMSIM_BF16, n, a, b, b)     # in place
    assert torch.equal(b, ref)


def test_edges(amd):
    import torch
    x = make(1000, "float32")
    assert torch.equal(amd.dropout(x, 0.0, seed=1), x)
    assert amd.dropout(x[:0], 0.5, seed=1).numel() == 0
    gone = ~torch.from_numpy(stays(1, 1000, 0.5, 0, 1)[0]).cuda()
    bad = torch.where(gone, torch.full_like(x, float("nan")), x)          # dropped elements may hold anything
    assert torch.equal(amd.dropout(bad, 0.5, seed=1), amd.dropout(x, 0.5, seed=1))
    bad = torch.where(gone, torch.full_like(x, float("inf")), x)
    assert torch.equal(amd.dropout(bad, 0.5, seed=1), amd.dropout(x, 0.5, seed=1))
    assert bool(torch.isnan(amd.dropout(torch.full_like(x, float("nan")), 0.5, seed=1)[~gone]).all())
    m = x.view(10, 100)
    assert torch.equal(amd.dropout(m, 0.5, seed=1), amd.dropout(x, 0.5, seed=1).view(10, 100))
    for bad_p in (-0.1, 1.0, float("nan"), 1.0 - 2.0 ** -40):
        with pytest.raises(amd.AmsimError):
            amd.dropout(x, bad_p, seed=1)
    with pytest.raises(ValueError):
        amd.dropout(m.t(), 0.5, seed=1)
    with pytest.raises(ValueError):
        amd.dropout(m, 0.5, seed=1, residual=x)
    with pytest.raises(TypeError):
        amd.dropout(m, 0.5, seed=1, residual=m.bfloat16())
    with pytest.raises(TypeError):
        amd.dropout(x.half(), 0.5, seed=1)
    with pytest.raises(TypeError):
        amd.dropout(x, 0.5, seed=1, step=torch.zeros(1, device="cuda"))


def test_share_that_stays(amd):
    """Of n elements n (1 - p) stay, to five deviations; other seeds, calls and steps give other masks."""
    import torch
    n = 1 << 22
    x = torch.ones(n, device="cuda")
    masks = []
    for p in (0.1, 0.37):
        for seed, call, step in ((1, 0, None), (2, 0, None), (1, 1, None), (1, 0, 2)):
            s = None if step is None else torch.tensor([step], device="cuda")
            m = amd.dropout(x, p, seed=seed, call=call, step=s) != 0
            assert abs(int(m.sum()) - n * (1 - p)) <= 5 * (n * p * (1 - p)) ** 0.5
            masks.append(m)
    for i in range(4):
        for j in range(i):
            both = int((masks[i] & masks[j]).sum())                       # independent: 0.81 n
            assert abs(both - n * 0.81) <= 5 * (n * 0.81 * 0.19) ** 0.5
    two = amd.dropout(x, 0.1, seed=1, call=2)
    assert torch.equal(masks[3], two != 0)                                # call + step


def test_captured_call_draws_by_its_step(amd):
    import torch
    x, step = make(9999, "float32"), torch.zeros(1, dtype=torch.int64, device="cuda")
    amd.dropout(x, 0.2, seed=3, step=step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = amd.dropout(x, 0.2, seed=3, call=10, step=step)
    for i in range(3):
        step.fill_(i)
        graph.replay()
        assert torch.equal(y, amd.dropout(x, 0.2, seed=3, call=10 + i))


def test_far_elements(amd):
    """Beyond 2^32 elements the quads' numbers and addresses keep all their bits."""
    import torch
    n = (1 << 32) + 4096 + 3
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = amd.dropout(x, 0.25, seed=9)
    first = (1 << 32) - 4096
    from philox_reference import quad_words
    w = quad_words(np.arange(first // 4, -(-n // 4), dtype=np.uint64), 0, 9).reshape(-1)[:n - first]
    assert np.array_equal((y[first:] != 0).cpu().numpy(), w >= round(0.25 * 2 ** 32))
