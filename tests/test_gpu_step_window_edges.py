"""c128_window_attention at the end of its table, with nothing to see, and what the rounding of its weights may do."""
import numpy as np
import pytest
import torch

import serving_ref as sref
from deepseek_v4_sparse_c128_gb300 import binding
from test_gpu_step_window import Case, consecutive

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def sums_of_rounded_weights(monkeypatch):
    """The shared tolerance counts a weight's rounding to bf16 in the sum over the entries. fp32 results are divided by the sum of the
    rounded weights, w'_j = w_j (1 + d_j), |d_j| <= 2^-8: sum w'_j k_j / sum w'_j differs from the result by
    (sum d_j w_j k_j - out sum d_j w_j) / (1 + ..), so by up to 2^-8 |out| more, which the tolerance of fp32
    results gets here. (bf16 results of short windows are not divided; those of long ones keep the shared tolerance.)"""
    monkeypatch.setattr(sref, "HALF_F32", sref.HALF_F32 + sref.HALF_BF16)


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


@pytest.mark.parametrize("H", [64, 16, 5])
@pytest.mark.parametrize("sink", [False, True], ids=["", "sink"])
@pytest.mark.parametrize("window,first", [(128, 4), (13, 0), (300, 4)])
def test_columns_that_all_entries_have_in_common(window, first, sink, H):
    """Columns 0 .. 191 are the same in every entry, so there the result is theirs, whatever the weights of the entries are and
    however these are rounded: times what the entries have of all weight, where there is a sink. (fp32 sums of at most 2^10 terms,
    which the tensor cores cut: 2^-23 of them each, 2^-13 at most and 2^-16 in earnest, as in the other tests; the factor of their
    sums and the sink's share 2^-20.)"""
    n = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    c = Case(93, consecutive(0, 5, n), [n + 5], H, window, first, 16, sink=sink, rubbish=False)
    flat = c.cache.reshape(len(c.cache), -1)
    for j in range(16):
        flat[:, j * 576:j * 576 + 192] = flat[0, :192]
        flat[:, 16 * 576 + 8 * j:16 * 576 + 8 * j + 3] = flat[0, 16 * 576:16 * 576 + 3]
    common = torch.from_numpy(c.entry(0, 0)[:192]).cuda()
    out, lse = c.run(torch.float32)
    assert binding.device_errors() == 0
    share = torch.ones_like(lse).double() if not sink else 1 - torch.exp(c.sink.cuda().double() - lse.double())
    want = share[..., None] * common
    # (lse is off by 2^-16, and so is the sink's share of it)
    tol = 2.0 ** -16 * want.abs() + (2.0 ** -20 + 2.0 ** -15 * (1 - share[..., None])) * common.abs()
    assert ((out[..., :192].double() - want).abs() <= tol).all()
    c.check(out, lse, tokens=range(0, n, 37))
