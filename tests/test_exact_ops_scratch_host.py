"""Scratch sizes of the exact operators (no GPU needed)."""
import pytest

import approximate_multiplier_dnn_gb300 as am


@pytest.fixture(scope="module", autouse=True)
def built():
    am.build()


def desc(tokens, vocab, dim, **kw):
    return am.VocabLossDesc(tokens=tokens, vocab=vocab, dim=dim, ignore_index=-100, reduction=am.AMSIM_REDUCE_MEAN, **kw)


@pytest.mark.parametrize("tokens,vocab,dim", [(1, 100, 16), (300, 8192, 256), (260, 5000, 64), (700, 1500, 136),
                                              (5000, 300, 1000)])
@pytest.mark.parametrize("which", [0, 1])
def test_least_scratch_is_the_least(tokens, vocab, dim, which):
    """A call that one chunk's scratch is enough for never needs more than it."""
    d = desc(tokens, vocab, dim)
    least, full = am.amsim_vocab_loss_workspace_min(d, which), am.amsim_vocab_loss_workspace_size(d, which)
    assert 0 < least <= full
