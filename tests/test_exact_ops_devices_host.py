"""The exact operators refuse tensors that are not on the current device (no GPU
needed: tensors of a second device are stood in for, and nothing may be
launched)."""
import pytest
import torch

import approximate_multiplier_dnn_gb300 as am


class On:
    """A contiguous tensor of some shape and type on a CUDA device."""
    is_cuda, device = True, "cpu"

    def __init__(self, index, *shape, dtype=torch.float32):
        self.index, self.shape, self.dtype, self.ndim = index, torch.Size(shape), dtype, len(shape)

    def get_device(self):
        return self.index

    def dim(self):
        return self.ndim

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def launched(monkeypatch):
    """The calls that reach the library; device 0 is the current one."""
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0
    monkeypatch.setattr(am, "lib", Library)
    monkeypatch.setattr(am, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(am, "_current_stream", lambda: 0)
    monkeypatch.setattr(am, "_ptr", lambda t: t.data_ptr() if hasattr(t, "data_ptr") else t)
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: On(0, *t.shape))
    return lambda: [c for c in calls if "workspace" not in c]


@pytest.mark.parametrize("off", range(5))
def test_block_norm(launched, off):
    x, y, p, q, gate = (On(int(i == off), *s) for i, s in enumerate([(4, 8), (4, 8), (8,), (8,), (1, 8)]))
    with pytest.raises(ValueError):
        am.block_norm(x, y, p, q, gate=gate)
    assert not launched()


@pytest.mark.parametrize("off", range(9))
def test_block_norm_backward(launched, off):
    shapes = [(4, 8)] * 4 + [(8,), (8,), (4,), (4,), (1, 8)]
    *args, gate = (On(int(i == off), *s) for i, s in enumerate(shapes))
    with pytest.raises(ValueError):
        am.block_norm_backward(*args, gate=gate)
    assert not launched()


@pytest.mark.parametrize("fn", ["vocab_loss", "vocab_loss_grad"])
@pytest.mark.parametrize("off", range(4))
def test_vocab_loss(launched, fn, off):
    kinds = [((4, 8), torch.bfloat16), ((50, 8), torch.bfloat16), ((4,), torch.int64), ((4,), torch.float32)]
    h, w, t, a = (On(int(i == off), *s, dtype=d) for i, (s, d) in enumerate(kinds))
    with pytest.raises(ValueError):
        getattr(am, fn)(h, w, t, row_weight=a)
    assert not launched()


def test_adamw(launched, monkeypatch):
    def entry(*index):
        return am.AdamwTensor.make(*(On(i, 8) for i in index))
    for off in range(4):
        with pytest.raises(ValueError):
            entry(*(int(i == off) for i in range(4)))
    here = am.adamw_table([entry(0, 0, 0, 0)])
    am.adamw_step(here, lr=1e-3, step=1)
    assert launched() == ["amsim_adamw_step"]
    with pytest.raises(ValueError):
        am.adamw_step(here, lr=1e-3, step=1, grad_scale=On(1, 1))
    monkeypatch.setattr(am, "_current_device", lambda: 1)
    with pytest.raises(ValueError):                          # the current device has changed since
        am.adamw_step(here, lr=1e-3, step=1)
    with pytest.raises(ValueError):
        am.adamw_table([here[0], entry(1, 1, 1, 1), e := entry(1, 1, 1, 1), _moved(e)])
    with pytest.raises(ValueError):
        am.adamw_moment_values(On(1, 8, dtype=torch.uint8), On(0, 1))
    assert launched() == ["amsim_adamw_step"]


def _moved(entry):
    copy = am.AdamwTensor()
    copy.device = entry.device + 1
    return copy


@pytest.mark.parametrize("shape", [(8, 2), (2, 2, 4), (4, 4), (1, 2, 8), (3, 8), (0, 8), (12,), ()])
def test_gate_of_another_shape(launched, shape):
    """As many values as a gate's, but no rows of channels: refused, not read as if they were."""
    x = On(0, 4, 8)
    with pytest.raises(ValueError):
        am.block_norm(x, x, gate=On(0, *shape))
    with pytest.raises(ValueError):
        am.block_norm_backward(x, None, x, x, None, None, None, None, gate=On(0, *shape))
    assert not launched()
