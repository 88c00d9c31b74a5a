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


@pytest.mark.parametrize("which", [0, 1])
def test_scratch_for_copies_only_where_they_are_made(which):
    """Operands that are read in place take no room; a base or a row stride off
    16 bytes, or many rows of h that are no whole lines, take a copy's."""
    P, tokens, vocab, dim = 1 << 20, 300, 50_000, 1000
    copy_h, copy_w = tokens * 1024 * 2, vocab * 1024 * 2
    both = am.amsim_vocab_loss_workspace_size(desc(tokens, vocab, dim), which)

    def at(d, h=P, w=P):
        return am.amsim_vocab_loss_workspace_size_at(d, which, h, w)
    none = at(desc(tokens, vocab, dim))
    assert both - none == -(-copy_h // 256) * 256 + copy_w
    assert at(desc(tokens, vocab, dim), P + 2, P) == at(desc(tokens, vocab, dim, ld_h=1001)) == both - copy_w
    assert at(desc(tokens, vocab, dim), P, P + 8) == at(desc(tokens, vocab, dim, ld_w=1004)) == none + copy_w
    assert at(desc(tokens, vocab, 1001)) == am.amsim_vocab_loss_workspace_size(desc(tokens, vocab, 1001), which)
    many = desc(2000, vocab, dim)
    assert at(many) == am.amsim_vocab_loss_workspace_size(many, which) - copy_w
    assert at(desc(2000, vocab, 1024)) == am.amsim_vocab_loss_workspace_size(desc(2000, vocab, 1024), which) - \
        2000 * 2048 - copy_w
    assert at(desc(0, vocab, dim)) == 0
