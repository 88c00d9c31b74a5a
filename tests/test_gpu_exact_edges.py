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
