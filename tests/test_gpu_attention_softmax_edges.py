"""The attention softmax where what is not seen is not finite."""
import pytest

from test_gpu_attention_softmax import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keys", [40, 90, 129, 300, 512, 1028, 1301, 40000, 40001])
@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("way", ["causal", "lengths", "behind the last key"])
def test_bias_that_only_hidden_keys_use(amd, keys, p, way):
    """NaN, infinities and any other number in the buckets of keys that a row
    does not see, or of places behind the last key, leave every result as it is."""
    import torch
    s, d, t, b = make(2, 2, 3, keys, keys, "both")
    n = torch.tensor([keys - 7, keys - 20], dtype=torch.int32, device="cuda")
    kw = {"causal": dict(causal=True, offset=keys // 2), "lengths": dict(lengths=n, offset=keys - 7),
          "behind the last key": dict(offset=keys - 1)}[way]
    kw.update(buckets=b, p=p, seed=3)
    if way == "behind the last key":         # one row, at the last key's place
        s, d = s[:, :, :1].contiguous(), d[:, :, :1].contiguous()

    def run(later):
        table = t.clone()
        table[16:] = later                   # the buckets of keys after the query's place
        probs, stats = amd.attention_softmax(s, table=table, **kw)
        ds, dt = amd.attention_softmax_backward(d, scores=s, stats=stats, table=table, **kw)
        return probs, stats, ds, dt
    want = run(0.0)
    assert all(bool(torch.isfinite(v).all()) for v in want) and not want[3][16:].any()
    for value in (float("nan"), float("inf"), -float("inf"), 3e38):
        for got, ref in zip(run(value), want):
            assert torch.equal(got, ref), f"{value}"
