"""What the attention softmax takes for its arguments (no GPU needed: nothing
is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import approximate_multiplier_dnn_gb300 as am
from test_between_ops_host import Tensor
from test_exact_ops_devices_host import launched  # noqa: F401  (a fixture)


@pytest.fixture
def described(launched, monkeypatch):  # noqa: F811
    """The descriptor that a call with this offset would make."""
    return lambda offset: am._softmax_call((2, 3, 4, 8), None, None, None, True, offset, 0.0, 0, 0, None, 0)


@pytest.mark.parametrize("offset", [7, np.int64(7), np.int32(-7), True, 1 << 40])
def test_offsets_are_whole_numbers_of_any_kind(described, offset):
    assert described(offset).offset == int(offset) and not described(offset).offsets


@pytest.mark.parametrize("offset", [7.0, np.float32(7), "7", None, [1, 2], np.zeros(2, np.int32)])
def test_other_offsets_are_refused(described, offset):
    with pytest.raises(TypeError):
        described(offset)


@pytest.mark.parametrize("offset", [1 << 63, (1 << 64) + 5, -(1 << 64), (1 << 40) + 1])
def test_offsets_that_no_cache_has_are_refused(described, offset):
    """Cut to 64 bits they would be other places."""
    with pytest.raises(ValueError):
        described(offset)


def test_offset_tensors(described):
    assert described(Tensor(0, 2, dtype=torch.int32)).offsets == 1 << 20
    for t, error in ((Tensor(0, 3, dtype=torch.int32), ValueError), (Tensor(0, 2, dtype=torch.int64), TypeError),
                     (Tensor(1, 2, dtype=torch.int32), ValueError)):
        with pytest.raises(error):
            described(t)


@pytest.mark.parametrize("bias", [dict(num_buckets=-1), dict(max_distance=-5), dict(max_distance=1 << 30)])
def test_sizes_of_a_bias_that_is_not_there_are_not_looked_at(bias):
    am.build()
    L, P = am.lib(), 1 << 20
    for size, status in ((0, am.AMSIM_OK), (2, None)):       # with rows a call gets as far as the device
        d = ctypes.byref(am.AttentionSoftmaxDesc(batch=size, heads=3, queries=4, keys=8, **bias))
        if size and torch.cuda.is_available():
            continue
        for rc in (L.amsim_attention_softmax_fwd(d, P, None, None, P, P, None),
                   L.amsim_attention_softmax_bwd(d, P, None, None, P, None, None, P, None, None, 0, None)):
            assert rc == status if status is not None else rc != am.AMSIM_EINVAL
        assert L.amsim_attention_softmax_fwd(d, P, P, P, P, P, None) in (am.AMSIM_EINVAL, am.AMSIM_EUNSUPPORTED)
