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


@pytest.fixture(autouse=True)
def sums_of_rounded_weights(monkeypatch):
    """The shared tolerance counts a weight's rounding to bf16 in the sum over the entries. fp32 results are divided by the sum of the
    rounded weights, w'_j = w_j (1 + d_j), |d_j| <= 2^-8: sum w'_j k_j / sum w'_j differs from the result by
    (sum d_j w_j k_j - out sum d_j w_j) / (1 + ..), so by up to 2^-8 |out| more, which the tolerance of fp32
    results gets here. (bf16 results of short windows are not divided; those of long ones keep the shared tolerance.)"""
    monkeypatch.setattr(sref, "HALF_F32", sref.HALF_F32 + sref.HALF_BF16)


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


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("name", WALKS)
def test_walk(name, kind):
    """All tokens of three CTAs, with a sink."""
    H, window, first, each, begin = WALKS[name]
    c = Walk(len(name) + 20, H, window, first, each, begin, sink=True)
    out, lse = c.walk(kind)
    assert binding.device_errors() == 0
    c.check_tokens(out, lse, c.of_ctas())
    # (of the others: that none was left out, and that no weight of 0 met what is not finite)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all() and not (out == 3).all(-1).any() and not (lse == 7).any()


@pytest.mark.parametrize("name", ["one_an_item", "two_an_item", "small_ring_five_heads", "no_room_few_heads", "much_room_few_heads", "group_of_37_heads"])
def test_queries_that_are_not_finite(name):
    """Their own row, and no other: not the token's other heads, nor the tokens beside it in the item and in the items around it."""
    H, window, first, each, begin = WALKS[name]
    c = Walk(len(name) + 40, H, window, first, each, begin)
    clean = [x.clone() for x in c.walk()]
    n = len(c.tokens)
    rows = [(t, (5 * t) % H) for t in range(7, n, 29)]
    for i, (t, h) in enumerate(rows):
        c.on_gpu[t, h, (31 * t) % 512] = float("nan") if i % 2 else float("inf")
    out, lse = c.walk()
    torch.cuda.synchronize()
    hit = torch.zeros(n, H, dtype=torch.bool, device="cuda")
    hit[[t for t, _ in rows], [h for _, h in rows]] = True
    nan = torch.zeros_like(hit)
    nan[[t for t, _ in rows[1::2]], [h for _, h in rows[1::2]]] = True
    assert torch.isnan(out[nan].float()).all() and torch.isnan(lse[nan]).all()
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("name", ["one_an_item", "two_an_item", "small_ring_two", "much_room_few_heads"])
@pytest.mark.parametrize("factor", [30.0, 1e-3, 2000.0])
def test_scores_of_any_size(name, factor):
    H, window, first, each, begin = WALKS[name]
    c = Walk(len(name) + 60, H, window, first, each, begin)
    c.on_gpu = (c.on_gpu.float() * factor).bfloat16()
    out, lse = c.walk()
    c.check_tokens(out, lse, c.of_ctas()[::2])


@pytest.mark.parametrize("name", ["one_an_item", "small_ring", "small_ring_two", "much_room_few_heads"])
def test_entries_of_any_magnitude_that_are_not_seen(name):
    """Entries so large that a score with them has no room, come and gone: tokens that do not see them are not touched."""
    H, window, first, each, begin = WALKS[name]
    c = Walk(len(name) + 80, H, window, first, each, begin)
    flat, n = c.cache.reshape(len(c.cache), -1), len(c.tokens)
    sees = torch.zeros(n, dtype=torch.bool)
    for j in range(max(first, begin) + 3, begin + n, 3 * window + 1):
        page, off = c.table[0, j // BLOCK], j % BLOCK
        flat[page, BLOCK * 576 + off * 8:BLOCK * 576 + off * 8 + 7] = 246  # 2^119
        flat[page, off * 576:off * 576 + 448] = 0x7e                      # 448
        sees[max(0, j - begin):j - begin + window] = True
    c.on_gpu = c.on_gpu.abs()
    out, lse = c.walk()
    assert 0 < sees.sum() < n
    assert torch.isfinite(out[~sees.cuda()].float()).all()
    c.check_tokens(out, lse, [t for t in c.of_ctas() + list(range(0, n, 61)) if not sees[t]])


@pytest.mark.parametrize("H,window,first", [(65, 300, 4), (128, 200, 0), (128, 137, 0), (17, 600, 2), (100, 1000, 140)])
def test_long_windows_of_many_heads(H, window, first):
    """Some hundred tokens, more than there are CTAs for their head groups; results and their parts of several groups."""
    tokens = consecutive(0, 150, 170) + consecutive(1, 0, 80) + [(2, 2500), (2, 7), (3, 900)] * 7
    c = Case(73 + H, tokens, [320, 80, 2501, 901], H, window, first, BLOCK, sink=True, skip=[0, 77, 200])
    for kind in (torch.bfloat16, torch.float32):
        out, lse = c.run(kind)
        assert binding.device_errors() == 0
        c.check(out, lse, tokens=[0, 77, 200, *range(1, len(tokens), 11), *range(250, len(tokens))])


@pytest.mark.parametrize("H", [128, 65, 16, 7])
def test_prompts_of_several_requests(H):
    """Prompts and parts of prompts, some tokens skipped, over CTAs of several tokens each; the same rows in another order."""
    n = 3 * sms()
    tokens = consecutive(0, 0, n) + consecutive(1, 500, n // 2) + [(2, 60)] + consecutive(3, 131, n // 3 + 1)
    lens = [n, 500 + n // 2, 61, 132 + n // 3]
    skip = [0, 1, n - 1, n, n + 40, n + 41, len(tokens) - 1]
    c = Case(74 + H, tokens, lens, H, 128, 4, 64, sink=True, skip=skip)
    out, lse = c.run()
    assert binding.device_errors() == 0
    c.check(out, lse, tokens=[*skip, *range(2, len(tokens), 23), *range(n - 9, n + 9)])
    order = np.random.default_rng(75).permutation(len(tokens))
    c.tokens, c.skip = [c.tokens[t] for t in order], {i for i, t in enumerate(order) if t in c.skip}
    c.q, c.req, c.pos, c.slots = c.q[order], c.req[order], c.pos[order], c.slots[order]
    out, lse = c.run()
    c.check(out, lse, tokens=[*sorted(c.skip), *range(0, len(tokens), 29)])


@pytest.mark.parametrize("H,each", [(64, 12), (128, 7), (5, 12)])
def test_a_table_with_rows_for_more_requests(H, each):
    """Whether tokens go over the CTAs in order, and which entries they share, does not depend on rows that no token is of: items of one
    token (of 64 heads and more all are) give the same bits. Padding, and tokens of requests that are not there, change nothing."""
    c = Walk(H, H, 128, 4, each, 300, sink=True)
    n = len(c.tokens)
    want = [x.clone() for x in c.walk()]
    c.check_tokens(*want, c.of_ctas())
    c.table = np.concatenate([c.table, np.full((n, c.table.shape[1]), -1, np.int32)])
    out, lse = c.walk()
    assert binding.device_errors() == 0
    if H >= 64:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    c.check_tokens(out, lse, c.of_ctas())
    c.req[5::9] = -1
    c.slots[3::7] = -1
    c.skip = {t for t in range(n) if t % 7 == 3 or t % 9 == 5}
    out, lse = c.walk()
    assert binding.device_errors() == 1
    left = torch.tensor([t in c.skip for t in range(n)], device="cuda")
    assert (out[left] == 3).all() and (lse[left] == 7).all()
    c.skip = set()
    c.check_tokens(out, lse, [t for t in c.of_ctas() if not left[t]])


def test_a_decode_step_with_a_few_drafts():
    """Tokens of which some follow one another, some do not: either way of dealing them out."""
    rng = np.random.default_rng(76)
    for follow in (0.2, 0.8):
        tokens, lens = [], []
        while len(tokens) < 3 * sms():
            p, k = int(rng.integers(0, 300)), 2 if rng.random() < follow else 1
            tokens += consecutive(len(lens), p, k)
            lens.append(p + k)
        lens += [1] * (2 * len(tokens))
        c = Case(77, tokens, lens, 9, 100, 4, BLOCK, sink=True, skip=[0, 50, len(tokens) - 1])
        out, lse = c.run()
        assert binding.device_errors() == 0
        c.check(out, lse)
