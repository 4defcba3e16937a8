"""c128_window_attention where its CTAs walk many tokens in order: entries that come one at a time, leave the window and have
their places taken by others; entries that are not finite on that way."""
import copy

import numpy as np
import pytest
import torch

import serving_ref as sref
from deepseek_v4_sparse_c128_gb300 import binding
from test_gpu_step_window import Case, consecutive

pytestmark = pytest.mark.gpu
BLOCK = 16


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


class Walk(Case):
    """One request's tokens from `begin` on, `each` to a CTA (in order, a whole number of them)."""

    def __init__(self, seed, H, window, first, each, begin=0, sink=False):
        rng = np.random.default_rng(seed)
        columns = sms() // -(-H // 64)
        self.each, self.begin, n = each, begin, each * columns
        self.tokens, self.H, self.window, self.first, self.block = consecutive(0, begin, n), H, window, first, BLOCK
        blocks = sref.cdiv(begin + n, BLOCK)
        self.cache = sref.make_cache(rng, blocks, BLOCK)
        self.table = rng.permutation(blocks).astype(np.int32)[None]
        self.most = blocks * BLOCK
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.on_gpu = (2 * torch.randn(n, H, 512, generator=g, device="cuda")).bfloat16()
        self.sink = torch.from_numpy(rng.standard_normal(H)).float() if sink else None
        self.scale, self.skip, self.keys = 512 ** -0.5, set(), {}
        self.req, self.slots = np.zeros(n, np.int32), np.full(n, 5, np.int64)
        self.pos = begin + np.arange(n, dtype=np.int64)

    def walk(self, kind=torch.bfloat16):
        return self.run(kind, q=self.on_gpu)

    def check_tokens(self, out, lse, tokens):
        some, at = copy.copy(self), torch.tensor(tokens, device="cuda")
        some.tokens, some.q = [self.tokens[t] for t in tokens], self.on_gpu[at].cpu()
        some.check(out[at], lse[at])

    def of_ctas(self):
        """The tokens of the first CTA, of one in the middle and of the last."""
        ctas = len(self.tokens) // self.each
        return [t for c in (0, ctas // 2, ctas - 1) for t in range(c * self.each, (c + 1) * self.each)]

    def spoil(self, entries):
        """Makes one value of each of these entries NaN or infinite, of another column and in another way each; true for the
        tokens that see one."""
        flat = self.cache.reshape(len(self.cache), -1)
        bad = torch.zeros(len(self.tokens), dtype=torch.bool, device="cuda")
        pos = torch.from_numpy(self.pos).cuda()
        for i, j in enumerate(entries):
            page, off, column = self.table[0, j // BLOCK], j % BLOCK, 37 * i % 512
            if column >= 448:
                flat[page, off * 576 + 448:off * 576 + 576].view(np.uint16)[column - 448] = (0x7f80, 0xffc0, 0xff80)[i % 3]
            elif i % 4 == 3:
                flat[page, BLOCK * 576 + off * 8 + column // 64] = 255
                flat[page, off * 576 + column] |= 0x70   # (a code of zero times 2^128 would be 0)
            else:
                flat[page, off * 576 + column] = 0x7f | (i & 1) << 7
            bad |= (pos >= j) & ((pos - j < self.window) | (j < self.first))
        return bad


# heads; window, first entries; tokens to a CTA; where they begin. One head group of one token an item (64), or items of two.
# (136 places: 128 + 4 leaves a ring of 132, of which 4 are free; 12 + 120 one of 16, so places are taken again within a walk;
# 126 + 10 none that is free, so an item waits for the results of the one before.)
WALKS = {
    "one_an_item": (64, 128, 4, 12, 200), "two_an_item": (16, 128, 4, 24, 0), "two_of_five_heads": (5, 128, 4, 26, 1000),
    "small_ring": (64, 12, 120, 40, 150), "small_ring_two": (16, 12, 120, 40, 0), "small_ring_five_heads": (5, 12, 120, 41, 300),
    "no_room": (64, 126, 10, 12, 0), "no_room_few_heads": (9, 126, 10, 25, 777), "much_room": (64, 7, 3, 30, 0),
    "much_room_few_heads": (3, 7, 3, 70, 5), "groups": (128, 128, 4, 12, 100), "group_of_one_head": (65, 100, 0, 9, 0),
    "group_of_37_heads": (101, 12, 120, 33, 130),
}


@pytest.mark.parametrize("name", WALKS)
def test_entries_that_are_not_finite(name):
    """Seen from a run's start, and come by one; their places are used again by entries that are."""
    H, window, first, each, begin = WALKS[name]
    c = Walk(len(name), H, window, first, each, begin)
    n = len(c.tokens)
    # every few windows one, in all phases of a CTA's walk; none among the first entries, which all tokens see
    step = 2 * window + 5
    step += step % each == 0
    bad = c.spoil([j for j in range(max(first, begin - window // 2), begin + n, step)])
    assert 0 < bad.sum() < n
    out, lse = c.walk()
    assert binding.device_errors() == 0
    assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    assert torch.isfinite(out[~bad].float()).all() and torch.isfinite(lse[~bad]).all()
    c.check_tokens(out, lse, [t for t in c.of_ctas() if not bad[t]] + [t for t in range(0, n, 61) if not bad[t]])


@pytest.mark.parametrize("name", ["one_an_item", "two_an_item", "small_ring_five_heads", "group_of_one_head"])
def test_first_entries_that_are_not_finite(name):
    H, window, first, each, begin = WALKS[name]
    first = max(first, 3)
    c = Walk(len(name), H, window, first, each, 0)
    bad = c.spoil([2])
    out, lse = c.walk()
    assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    assert bad[2:].all() and not bad[:2].any()
    c.check_tokens(out, lse, [0, 1])


@pytest.mark.parametrize("H", [64, 5])
def test_a_column_of_each_entry_that_a_run_begins_with(H):
    """Requests of one token each, several to a CTA: one value of one of its entries is NaN in every other, another place and another
    column each, and the request behind it sees a few entries only, so that the others' places stay."""
    n = 6 * sms()
    rng = np.random.default_rng(70)
    lens = [132 if i // sms() % 2 == 0 else 1 + i % 7 for i in range(n)]
    tokens = [(r, m - 1) for r, m in enumerate(lens)]
    c = Case(71, tokens, lens, H, 128, 4, BLOCK, rubbish=False)
    flat = c.cache.reshape(len(c.cache), -1)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    for r in range(n):
        if lens[r] < 132:
            continue
        j, column = int(rng.integers(132)), int(rng.integers(512))
        page, off = c.table[r, j // BLOCK], j % BLOCK
        if column < 448:
            flat[page, off * 576 + column] = 0xff
        else:
            flat[page, off * 576 + 448:off * 576 + 576].view(np.uint16)[column - 448] = 0x7fc0
        bad[r] = True
    out, lse = c.run()
    assert binding.device_errors() == 0
    assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    c.check(out, lse, tokens=[t for t in range(n) if not bad[t]])


@pytest.mark.parametrize("H", [16, 5, 1])
def test_a_run_whose_oldest_entry_is_not_finite(H):
    """Only a run's first token sees the entry; the tokens beside it in the item do not."""
    each, window = 4, 12
    n = 4 * sms()
    lens = [40 + each] * n
    tokens = [t for r in range(n) for t in consecutive(r, 40, each)]
    c = Case(72, tokens, lens, H, window, 2, BLOCK, rubbish=False)
    flat = c.cache.reshape(len(c.cache), -1)
    oldest = 40 - window + 1
    for r in range(0, n, 3):
        page, off, column = c.table[r, oldest // BLOCK], oldest % BLOCK, 11 * r % 448
        flat[page, off * 576 + column] = 0x7f
    bad = torch.tensor([r % 3 == 0 and p == 40 for r, p in tokens], device="cuda")
    out, lse = c.run()
    assert binding.device_errors() == 0
    assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    assert torch.isfinite(out[~bad].float()).all()
    c.check(out, lse, tokens=[t for t in range(0, len(tokens), 7) if not bad[t]])
