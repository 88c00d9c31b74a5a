"""A table has one owner: copies of a Lut, or of a layer that holds one, are
that owner's (no GPU needed)."""
import copy
import gc
import pickle

import pytest
import torch

import approximate_multiplier_dnn_gb300 as am
from approximate_multiplier_dnn_gb300 import layers


class Table(am.Lut):
    """A Lut of no library's: closing one writes its handle down."""
    freed = []

    def close(self):
        if self.handle:
            self.freed.append(self.handle)
            self.handle = None


@pytest.fixture
def freed():
    """The handles that were freed."""
    Table.freed.clear()
    return Table.freed


def test_copies_free_nothing(freed):
    """A copy that is dropped left its original, and other copies, with a freed
    table, and freed it again at each one's end."""
    lut = Table(4096, 7)
    copies = [copy.copy(lut), copy.deepcopy(lut), copy.deepcopy([lut, lut])]
    net = torch.nn.ModuleList([layers.AMDense(4, 4, lut, device="cpu"), layers.AMAttention(lut)])
    copies.append(copy.deepcopy(net))
    assert copies[-1][0].lut is lut and copies[-1][0].weight is not net[0].weight
    del copies
    gc.collect()
    assert not freed and lut.handle == 4096
    del lut
    gc.collect()
    assert not freed                                                      # the layers still hold it
    del net
    gc.collect()
    assert freed == [4096]


def test_pickling_is_refused(freed):
    """A handle means nothing in another process, and in this one would be freed twice."""
    lut = Table(4096, 7)
    for what in (lut, layers.AMAttention(lut)):
        with pytest.raises(TypeError, match="Lut"):
            pickle.dumps(what)
    layers.AMAttention(lut, dropout=0.1).state_dict()                     # holds no table
    lut.close()
    assert freed == [4096]
