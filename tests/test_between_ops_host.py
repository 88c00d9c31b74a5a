"""Host-side checks of the operators between two contractions (no GPU needed):
every refusal comes back before any device work, sizes are reported, the
binding's structs have the header's layout, the buckets of distances, and
tensors of another device."""
import ctypes
import math
import subprocess

import pytest
import torch

import approximate_multiplier_dnn_gb300 as am
from test_exact_ops_devices_host import On, launched  # noqa: F401  (launched is a fixture)

P = 1 << 20          # an aligned address that is never read: each call below is refused first
EINVAL = am.AMSIM_EINVAL


@pytest.fixture(scope="module")
def L():
    am.build()
    return am.lib()


def drop(L, d=am.DropoutDesc(0.1, 1, 2, None), type=0, n=8, x=P, r=None, y=P):
    return L.amsim_dropout(ctypes.byref(d) if d else None, type, n, x, r, y, None)


def test_dropout_rejects(L):
    assert drop(L, None) == EINVAL
    for p in (-0.5, 1.0, 2.0, math.nan, math.inf, 1 - 2.0 ** -40):
        assert drop(L, am.DropoutDesc(p, 1, 2, None)) == EINVAL
    assert drop(L, am.DropoutDesc(0.1, 1, 2, P + 4)) == EINVAL
    for bad in (dict(type=2), dict(type=-1), dict(n=-1), dict(x=None), dict(y=None), dict(x=P + 2), dict(y=P + 1),
                dict(r=P + 2), dict(type=1, r=P + 1), dict(n=1 << 62)):
        assert drop(L, **bad) == EINVAL
    assert drop(L, n=0, x=None, y=None) == am.AMSIM_OK


def soft(**kw):
    d = dict(batch=2, heads=3, queries=4, keys=8, num_buckets=32, max_distance=128)
    d.update(kw)
    return am.AttentionSoftmaxDesc(**d)


def fwd(L, d, s=P, t=P, b=P, probs=P, stats=P):
    return L.amsim_attention_softmax_fwd(ctypes.byref(d) if d else None, s, t, b, probs, stats, None)


def bwd(L, d, g=P, s=None, st=None, probs=P, t=None, b=P, ds=P, dt=P, ws=P, n=1 << 20):
    return L.amsim_attention_softmax_bwd(ctypes.byref(d) if d else None, g, s, st, probs, t, b, ds, dt, ws, n, None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(heads=-1), dict(queries=-1), dict(keys=-1), dict(keys=1 << 31),
                                 dict(batch=1 << 20, queries=1 << 20), dict(ld_scores=7), dict(ld_probs=-8),
                                 dict(ld_dprobs=7), dict(ld_dscores=1), dict(ld_scores=1 << 32), dict(causal=2),
                                 dict(causal=-1), dict(reserved=1), dict(lengths=P + 2), dict(offsets=P + 1),
                                 dict(offset=1 << 41), dict(num_buckets=-1), dict(max_distance=-1),
                                 dict(dropout=am.DropoutDesc(1.0, 0, 0, None)),
                                 dict(dropout=am.DropoutDesc(0.1, 0, 0, P + 4))])
def test_attention_softmax_rejects_descriptors(L, bad):
    assert fwd(L, soft(**bad)) == EINVAL and bwd(L, soft(**bad)) == EINVAL
    assert L.amsim_attention_softmax_workspace_size(ctypes.byref(soft(**bad))) == 0


def test_attention_softmax_rejects_arguments(L):
    d = soft()
    assert fwd(L, None) == EINVAL and bwd(L, None) == EINVAL
    for bad in (dict(s=None), dict(probs=None), dict(t=None), dict(b=None), dict(s=P + 1), dict(stats=P + 2),
                dict(t=P + 2), dict(b=P + 3), dict(probs=P + 2)):
        assert fwd(L, d, **bad) == EINVAL
    assert fwd(L, soft(num_buckets=0)) == EINVAL
    assert fwd(L, soft(max_distance=am.AMSIM_MAX_DISTANCE + 1)) == am.AMSIM_EUNSUPPORTED
    for bad in (dict(g=None), dict(ds=None), dict(probs=None), dict(s=P, st=P), dict(probs=None, s=P), dict(b=None),
                dict(t=P), dict(g=P + 2), dict(ds=P + 1), dict(dt=P + 2), dict(ws=P + 1)):
        assert bwd(L, d, **bad) == EINVAL
    assert bwd(L, soft(dropout=am.DropoutDesc(0.1, 0, 0, None))) == EINVAL             # dropped probabilities
    assert bwd(L, soft(max_distance=am.AMSIM_MAX_DISTANCE + 1)) == am.AMSIM_EUNSUPPORTED
    for none in (dict(batch=0), dict(heads=0), dict(queries=0), dict(keys=0)):
        assert fwd(L, soft(**none), s=None, probs=None, stats=None) == am.AMSIM_OK
        assert bwd(L, soft(**none), g=None, probs=None, ds=None, dt=None, ws=None, n=0) == am.AMSIM_OK
        assert L.amsim_attention_softmax_workspace_size(ctypes.byref(soft(**none))) == 0


def norm(**kw):
    d = dict(batch=2, pixels=4, channels=8, groups=2, eps=1e-5)
    d.update(kw)
    return am.GroupNormDesc(**d)


def gfwd(L, d, x=P, w=P, b=P, y=P, mean=P, rstd=P, ws=P, n=1 << 30):
    return L.amsim_group_norm_fwd(ctypes.byref(d) if d else None, x, w, b, y, mean, rstd, ws, n, None)


def gbwd(L, d, dy=P, x=P, w=P, b=P, mean=P, rstd=P, dx=P, dw=P, db=P, ws=P, n=1 << 30):
    return L.amsim_group_norm_bwd(ctypes.byref(d) if d else None, dy, x, w, b, mean, rstd, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(pixels=-1), dict(channels=0), dict(groups=0), dict(groups=3),
                                 dict(groups=-2), dict(ldx=7), dict(ldy=-8), dict(lddx=7), dict(x_type=2), dict(y_type=-1),
                                 dict(activation=3), dict(activation=-1), dict(eps=-1.0), dict(eps=math.nan),
                                 dict(eps=math.inf), dict(batch=1 << 31), dict(pixels=1 << 41), dict(channels=1 << 25)])
def test_group_norm_rejects_descriptors(L, bad):
    assert gfwd(L, norm(**bad)) == EINVAL and gbwd(L, norm(**bad)) == EINVAL
    assert [L.amsim_group_norm_workspace_size(ctypes.byref(norm(**bad)), i) for i in (0, 1)] == [0, 0]


def test_group_norm_rejects_arguments(L):
    d = norm()
    assert gfwd(L, None) == EINVAL and gbwd(L, None) == EINVAL
    for bad in (dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None), dict(x=P + 2), dict(y=P + 1), dict(w=P + 2),
                dict(b=P + 1), dict(mean=P + 2), dict(rstd=P + 3), dict(ws=P + 4)):
        assert gfwd(L, d, **bad) == EINVAL
    for bad in (dict(x=None), dict(dy=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(dx=P + 2),
                dict(dy=P + 1), dict(dw=P + 2), dict(db=P + 1), dict(ws=P + 4)):
        assert gbwd(L, d, **bad) == EINVAL
    for which, call in ((0, gfwd), (1, gbwd)):
        size = L.amsim_group_norm_workspace_size(ctypes.byref(d), which)
        if size:
            assert call(L, d, n=size - 1) == EINVAL and call(L, d, ws=None) == EINVAL
    assert L.amsim_group_norm_workspace_size(ctypes.byref(d), 2) == 0
    assert gfwd(L, norm(batch=0), x=None, y=None, mean=None, rstd=None, ws=None, n=0) == am.AMSIM_OK
    assert gbwd(L, norm(batch=0), x=None, dy=None, dx=None, dw=None, db=None, ws=None, n=0) == am.AMSIM_OK


def test_struct_layouts_match_header(tmp_path):
    structs = {"amsim_dropout_desc": am.DropoutDesc, "amsim_attention_softmax_desc": am.AttentionSoftmaxDesc,
               "amsim_group_norm_desc": am.GroupNormDesc}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "amsim.h"', "int main(void) {"]
    want = []
    for name, cls in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    lines += ['printf("%d %d %d %d\\n", AMSIM_MAX_DISTANCE, AMSIM_ACT_NONE, AMSIM_ACT_RELU, AMSIM_ACT_SILU);',
              "return 0; }"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c11", f"-I{str(am.HEADER).rsplit('/', 1)[0]}", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == want + [am.AMSIM_MAX_DISTANCE, *am.ACTIVATIONS.values()]


@pytest.mark.parametrize("both", [True, False])
@pytest.mark.parametrize("buckets,distance", [(32, 128), (8, 20), (64, 800), (6, 1000), (4, 5)])
def test_relative_buckets(both, buckets, distance):
    """One distance a bucket near the query, then ranges that grow by a constant
    factor, in 64 bits away from their edges; exact powers fall into the bucket they begin."""
    b = am.relative_buckets(buckets, distance, both).tolist()
    count = buckets // 2 if both else buckets
    near = count // 2
    assert len(b) == 2 * distance + 1 and max(b) < buckets and min(b) >= 0
    for d in range(-distance, distance + 1):
        got, far = b[d + distance], abs(d) if both else max(0, -d)
        if both and d > 0:
            got -= count
        if far < near:
            assert got == far
            continue
        k = near + math.log(far / near) / math.log(distance / near) * (count - near)
        assert got == min(count - 1, round(k) if abs(k - round(k)) < 1e-9 else int(k))


def test_conveniences_reject_cpu_tensors():
    x = torch.zeros(2, 3, 4, 8)
    for call in (lambda: am.dropout(x, 0.1, seed=1), lambda: am.attention_softmax(x), lambda: am.group_norm(x, 2),
                 lambda: am.attention_softmax_backward(x, probs=x),
                 lambda: am.group_norm_backward(x, x, None, None, torch.zeros(2, 2), torch.zeros(2, 2))):
        with pytest.raises(TypeError):
            call()


class Tensor(On):
    def stride(self, i=None):
        s, at = [], 1
        for n in reversed(self.shape):
            s.insert(0, at)
            at *= n
        return tuple(s) if i is None else s[i]


@pytest.mark.parametrize("off", range(3))
def test_dropout_on_another_device(launched, off):  # noqa: F811
    x, r, step = (Tensor(int(i == off), *s, dtype=t) for i, (s, t) in enumerate(
        [((4, 8), torch.float32), ((4, 8), torch.float32), ((1,), torch.int64)]))
    with pytest.raises(ValueError):
        am.dropout(x, 0.1, seed=1, step=step, residual=r)
    assert not launched()


@pytest.mark.parametrize("off", range(9))
def test_attention_softmax_on_another_device(launched, off):  # noqa: F811
    shape = (2, 3, 4, 8)
    kinds = [(shape, torch.float32), ((32, 3), torch.float32), ((257,), torch.int32), ((2,), torch.int32),
             ((2,), torch.int32), (shape, torch.float32), (shape, torch.float32), ((2, 3, 4, 2), torch.float32),
             ((1,), torch.int64)]
    s, t, b, n, o, out, d, stats, step = (Tensor(int(i == off), *k, dtype=t) for i, (k, t) in enumerate(kinds))
    kw = dict(table=t, buckets=b, lengths=n, offset=o, out=out, p=0.1, step=step)
    if off not in (6, 7):
        with pytest.raises(ValueError):
            am.attention_softmax(s, **kw)
    with pytest.raises(ValueError):
        am.attention_softmax_backward(d, scores=s, stats=stats, **kw)
    assert not launched()


@pytest.mark.parametrize("off", range(6))
def test_group_norm_on_another_device(launched, off):  # noqa: F811
    kinds = [(2, 4, 8), (8,), (8,), (2, 4, 8), (2, 2), (2, 2)]
    x, w, b, dy, mean, rstd = (Tensor(int(i == off), *k) for i, k in enumerate(kinds))
    if off < 3:
        with pytest.raises(ValueError):
            am.group_norm(x, 2, w, b)
    with pytest.raises(ValueError):
        am.group_norm_backward(dy, x, w, b, mean, rstd)
    assert not launched()
