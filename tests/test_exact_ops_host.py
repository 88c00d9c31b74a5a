"""Host-side checks of the exact operators' entry points (no GPU needed): every
refusal comes back before any device work, sizes are reported, and the
binding's structs have the header's layout."""
import ctypes
import math
import subprocess

import pytest

import approximate_multiplier_dnn_gb300 as am

P = 1 << 20          # an aligned address that is never read: each call below is refused first


@pytest.fixture(scope="module")
def L():
    am.build()
    return am.lib()


def norm_desc(**kw):
    d = dict(rows=4, cols=16, alpha=1.0, eps=1e-6)
    d.update(kw)
    return am.BlockNormDesc(**d)


def norm_fwd(L, d, x=P, y=P, gate=None, w_post=P, w_pre=P, r=P, n=P):
    return L.amsim_block_norm_fwd(ctypes.byref(d) if d is not None else None, x, y, gate, w_post, w_pre, r, n, None,
                                  None, None)


def norm_bwd(L, d, dr=P, dn=P, r=P, y=P, gate=None, w_post=P, w_pre=P, sp=P, sq=P, dx=P, dy=P, dgate=None, dwp=P,
             dwq=P, ws=None, n=0):
    return L.amsim_block_norm_bwd(ctypes.byref(d), dr, dn, r, y, gate, w_post, w_pre, sp, sq, dx, dy, dgate, dwp, dwq,
                                  ws, n, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=0), dict(gate_rows=3), dict(gate_rows=-1), dict(x_type=2),
                                 dict(y_type=-1), dict(n_type=7), dict(ldx=15), dict(ldy=-16), dict(lddx=3),
                                 dict(alpha=math.inf), dict(alpha=math.nan), dict(eps=-1.0), dict(eps=math.nan)])
def test_block_norm_rejects_descriptors(L, bad):
    assert norm_fwd(L, norm_desc(**bad)) == am.AMSIM_EINVAL
    assert norm_bwd(L, norm_desc(**bad)) == am.AMSIM_EINVAL
    assert L.amsim_block_norm_workspace_size(ctypes.byref(norm_desc(**bad))) == 0


def test_block_norm_rejects_arguments(L):
    d = norm_desc()
    assert norm_fwd(L, None) == am.AMSIM_EINVAL
    assert norm_fwd(L, norm_desc(cols=am.AMSIM_BLOCK_NORM_MAX_COLS + 1)) == am.AMSIM_EUNSUPPORTED
    assert norm_fwd(L, d, x=None) == am.AMSIM_EINVAL
    assert norm_fwd(L, d, r=None, n=None) == am.AMSIM_EINVAL
    assert norm_fwd(L, d, y=None) == am.AMSIM_EINVAL                      # w_post without y
    assert norm_fwd(L, d, y=None, w_post=None, gate=P) == am.AMSIM_EINVAL
    assert norm_fwd(L, d, x=P + 2) == am.AMSIM_EINVAL                     # fp32 off its alignment
    assert norm_fwd(L, d, w_pre=P + 1) == am.AMSIM_EINVAL
    assert norm_fwd(L, norm_desc(rows=0)) == am.AMSIM_OK
    assert norm_bwd(L, d, dr=None, dn=None, dwq=None) == am.AMSIM_EINVAL
    assert norm_bwd(L, d, r=None) == am.AMSIM_EINVAL
    assert norm_bwd(L, d, sq=None) == am.AMSIM_EINVAL
    assert norm_bwd(L, d, sp=None) == am.AMSIM_EINVAL
    assert norm_bwd(L, d, dgate=P) == am.AMSIM_EINVAL                     # no gate
    assert norm_bwd(L, d, w_post=None) == am.AMSIM_EINVAL                 # dw_post without w_post
    assert norm_bwd(L, d, dn=None) == am.AMSIM_EINVAL                     # dw_pre without dn
    assert norm_bwd(L, d, y=None) == am.AMSIM_EINVAL
    assert norm_bwd(L, d, dx=None, dy=None, dwp=None, dwq=None) == am.AMSIM_EINVAL


def loss_desc(**kw):
    d = dict(tokens=4, vocab=100, dim=16, ignore_index=-100, reduction=am.AMSIM_REDUCE_MEAN)
    d.update(kw)
    return am.VocabLossDesc(**d)


def grad(L, d, h=P, w=P, t=P, rw=None, loss=P, dh=P, dw=P, ws=P, n=1 << 30):
    return L.amsim_vocab_loss_grad(ctypes.byref(d) if d is not None else None, h, w, t, rw, loss, None, None, dh, dw,
                                   ws, n, None)


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(vocab=0), dict(dim=0), dict(ld_h=15), dict(ld_dw=8),
                                 dict(ld_w=-16), dict(reduction=2)])
def test_vocab_loss_rejects_descriptors(L, bad):
    d = loss_desc(**bad)
    assert grad(L, d) == am.AMSIM_EINVAL
    assert L.amsim_vocab_loss(ctypes.byref(d), P, P, P, None, P, None, None, P, 1 << 30, None) == am.AMSIM_EINVAL
    for which in (0, 1):
        assert L.amsim_vocab_loss_workspace_size(ctypes.byref(d), which) == 0
        assert L.amsim_vocab_loss_workspace_min(ctypes.byref(d), which) == 0


@pytest.mark.parametrize("bad", [dict(h=None), dict(w=None), dict(t=None), dict(loss=None), dict(dh=None),
                                 dict(dw=None), dict(ws=None), dict(h=P + 1), dict(t=P + 4), dict(rw=P + 2),
                                 dict(ws=P + 16)])
def test_vocab_loss_rejects_arguments(L, bad):
    assert grad(L, loss_desc(), **bad) == am.AMSIM_EINVAL
    assert grad(L, None) == am.AMSIM_EINVAL


def test_vocab_loss_workspace(L):
    """More tokens never need a larger least scratch than the chunk, the fast
    size is at least the least one, and the gradients' exponentials are capped."""
    for which in (0, 1):
        least = [am.amsim_vocab_loss_workspace_min(loss_desc(tokens=t, vocab=5000), which) for t in (1, 128)]
        assert 0 < least[0] <= least[1]
        d = loss_desc(tokens=100_000, vocab=131072, dim=256)
        assert am.amsim_vocab_loss_workspace_size(d, which) >= am.amsim_vocab_loss_workspace_min(d, which) > 0
    d = loss_desc(tokens=1 << 20, vocab=131072, dim=64)
    assert am.amsim_vocab_loss_workspace_size(d, 1) < 6 << 30
    assert am.amsim_vocab_loss_workspace_size(d, 2) == 0
    assert am.amsim_vocab_loss_workspace_size(loss_desc(tokens=0), 1) == 0


def adam(**kw):
    t = dict(p=P, g=P, m=P, v=P, n=8, lr_scale=1.0)
    t.update(kw)
    return am.AdamwTensor(**t)


def step(L, tensors, **kw):
    h = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1)
    h.update(kw)
    arr = (am.AdamwTensor * max(1, len(tensors)))(*tensors)
    return L.amsim_adamw_step(len(tensors), arr, ctypes.byref(am.AdamwHyper(**h)), None)


@pytest.mark.parametrize("bad", [dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(n=-1), dict(g_type=3),
                                 dict(reserved=1), dict(m_scale=P), dict(v_scale=P), dict(p=P + 2), dict(g=P + 1),
                                 dict(copy=P + 1), dict(lr_scale=math.nan), dict(weight_decay=math.inf),
                                 dict(m=P + 1)])
def test_adamw_rejects_tensors(L, bad):
    assert step(L, [adam(**bad)]) == am.AMSIM_EINVAL


@pytest.mark.parametrize("bad", [dict(lr=math.nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
                                 dict(beta2=math.nan), dict(eps=-1e-8), dict(eps=math.inf), dict(step=0),
                                 dict(grad_scale=P + 2)])
def test_adamw_rejects_hyperparameters(L, bad):
    assert step(L, [adam()], **bad) == am.AMSIM_EINVAL


def test_adamw_rejects_mixed_moments_and_null(L):
    assert step(L, [adam(), adam(m_scale=P, v_scale=P)]) == am.AMSIM_EINVAL
    assert L.amsim_adamw_step(1, None, ctypes.byref(am.AdamwHyper()), None) == am.AMSIM_EINVAL
    assert L.amsim_adamw_step(1, (am.AdamwTensor * 1)(adam()), None, None) == am.AMSIM_EINVAL
    assert L.amsim_adamw_step(-1, None, ctypes.byref(am.AdamwHyper()), None) == am.AMSIM_EINVAL
    assert step(L, []) == am.AMSIM_OK                                     # nothing to do
    assert step(L, [am.AdamwTensor(n=0)]) == am.AMSIM_OK
    assert L.amsim_adamw_moment_values(None, P, 0, 4, P, None) == am.AMSIM_EINVAL
    assert L.amsim_adamw_moment_values(P, P, 0, -4, P, None) == am.AMSIM_EINVAL
    assert L.amsim_adamw_moment_values(None, None, 0, 0, None, None) == am.AMSIM_OK


def test_struct_layouts_match_header(tmp_path):
    structs = {"amsim_block_norm_desc": am.BlockNormDesc, "amsim_vocab_loss_desc": am.VocabLossDesc,
               "amsim_adamw_tensor": am.AdamwTensor, "amsim_adamw_hyper": am.AdamwHyper}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "amsim.h"', "int main(void) {"]
    want = []
    for name, cls in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    lines += [f'printf("%d %d\\n", AMSIM_ADAMW_BLOCK, AMSIM_BLOCK_NORM_MAX_COLS);', "return 0; }"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    inc = str(am.HEADER).rsplit("/", 1)[0]
    subprocess.run(["gcc", "-std=c11", f"-I{inc}", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == want + [am.AMSIM_ADAMW_BLOCK, am.AMSIM_BLOCK_NORM_MAX_COLS]


def test_conveniences_reject_cpu_and_odd_tensors():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        am.block_norm(x)
    with pytest.raises(ValueError):
        am.block_norm(torch.zeros(4))
    with pytest.raises(TypeError):
        am.vocab_loss(x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        am.vocab_loss(torch.zeros(4), x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        am.AdamwTensor.make(x, x, x, x)
    with pytest.raises(TypeError):
        am.adamw_moment_values(torch.zeros(4), torch.zeros(1))
    assert len(am.adamw_table([])) == 0
