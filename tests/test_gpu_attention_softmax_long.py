"""The attention softmax over many long rows, as the other tests count its
errors: clusters of blocks that each take several rows in turn, with the row in
registers or read twice, on and off 16 bytes, and one cluster a row."""
import pytest

from test_gpu_attention_softmax import both_ways, make

pytestmark = pytest.mark.gpu


def in_place(amd, s, d, probs, stats, **kw):
    """Written over what was read: the same bits."""
    import torch
    t, p = s.clone(), kw.get("p", 0.0)
    assert amd.attention_softmax(t, out=t, **kw)[0] is t and torch.equal(t, probs)
    way = dict(scores=s, stats=stats) if p else dict(probs=probs)
    want = amd.attention_softmax_backward(d, **way, **kw)
    for over in (d.clone(), next(iter(way.values())).clone()):
        if over.shape == d.shape:
            src = dict(way)
            if torch.equal(over, d):
                got = amd.attention_softmax_backward(over, out=over, **src, **kw)
            else:
                src[next(iter(src))] = over
                got = amd.attention_softmax_backward(d, out=over, **src, **kw)
            assert got[0] is over and torch.equal(over, want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("keys", [131072, 131075])
def test_single_tokens_of_a_long_cache(amd, keys):
    """Two sequences of 16 heads, each at its own place, with a bias."""
    import torch
    s, d, t, b = make(2, 16, 1, keys, 1, "past", buckets=8)
    n = torch.tensor([keys, keys // 3], dtype=torch.int32, device="cuda")
    both_ways(amd, s, d, t, b, lengths=n, offset=n - 1, causal=True)


# read twice by clusters of eight blocks (480 rows); the row in the registers of a cluster of two, forward (700 rows of
# 16387 keys) and backward (420 of 13001)
@pytest.mark.parametrize("queries,keys", [(480, 40000), (480, 40001), (700, 16387), (700, 16388), (420, 13000), (420, 13001)])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_many_rows(amd, queries, keys, p):
    s, d, t, b = make(1, 1, queries, keys, keys, "both", buckets=8)
    probs, stats = both_ways(amd, s, d, t, b, p=p, offset=keys // 2)
    in_place(amd, s, d, probs, stats, table=t, buckets=b, p=p, seed=77, call=5, offset=keys // 2)


@pytest.mark.parametrize("queries,keys", [(160, 40001), (300, 16388)])
def test_many_rows_that_see_some_keys(amd, queries, keys):
    """Causal rows of several heads and sequences, one of length zero, whose clusters go from one to the next."""
    import torch
    s, d, t, b = make(3, 2, queries, keys, 3, "past", buckets=8)
    n = torch.tensor([keys, 0, keys // 2], dtype=torch.int32, device="cuda")
    both_ways(amd, s, d, t, b, p=0.1, causal=True, lengths=n, offset=keys // 4)
