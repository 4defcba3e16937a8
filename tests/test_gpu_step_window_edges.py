"""c128_window_attention at the end of its table, and with nothing to see."""
import numpy as np
import pytest
import torch

from deepseek_v4_sparse_c128_gb300 import binding
from test_gpu_step_window import Case, consecutive

pytestmark = pytest.mark.gpu


def fill_all_places():
    """A call that leaves an entry in all 136 places of every SM's shared memory."""
    n = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    c = Case(90, [(r, 135) for r in range(n)], [136] * n, 3, 100, 36, 8)
    c.run()


@pytest.mark.parametrize("H", [1, 64, 20])
@pytest.mark.parametrize("sink", [False, True], ids=["", "sink"])
@pytest.mark.parametrize("most,block,window,first", [(64, 64, 36, 100), (64, 16, 1, 135), (3, 1, 7, 4), (128, 64, 6, 130), (0, 4, 5, 1), (0, 64, 120, 2)])
def test_first_entries_that_the_table_does_not_hold(most, block, window, first, sink, H):
    """More first entries than a row of the table holds: the tokens behind its end see those that there are."""
    fill_all_places()
    behind = [most, most + 1, first, first + 1, most + window - 1, most + window, 1000, 1 << 40, (1 << 63) - 1]
    tokens = consecutive(0, 0, min(most, 20)) + consecutive(0, max(0, most - 3), 5) + [(0, p) for p in behind]
    c = Case(91, tokens, [max(most, 1)], H, window, first, block, sink=sink, rubbish=False)
    c.table, c.most = c.table[:, :most // block].copy(), most
    c.pos = np.array([p for _, p in tokens], np.int64)
    out, lse = c.run()
    assert binding.device_errors() == 2  # positions behind the table
    c.check(out, lse)


@pytest.mark.parametrize("sink", [False, True], ids=["", "sink"])
def test_nothing_to_see_has_the_sink_as_its_lse(sink):
    """A table without columns, first entries or not: zeros, and an lse of the sink."""
    fill_all_places()
    for first in (0, 1, 2, 16):
        c = Case(92, [(0, 0), (0, 5), (0, 300)], [64], 9, 20, first, 64, sink=sink, rubbish=False)
        c.table, c.most = c.table[:, :0], 0
        out, lse = c.run()
        assert binding.device_errors() == 2
        assert (out == 0).all()
        if sink:  # kept times log2(e) and given times log(2): two rounded constants, two products, half a step each
            assert ((lse - c.sink.cuda()).abs() <= 2.0 ** -22 * c.sink.cuda().abs()).all()
        else:
            assert (lse == -np.inf).all()
