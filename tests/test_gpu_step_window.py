"""c128_window_attention on the GPU against a reference in 64 bits, one token at a time."""
import numpy as np
import pytest
import torch

import serving_ref as sref
import step_ref as ref
from deepseek_v4_sparse_c128_gb300 import binding

pytestmark = pytest.mark.gpu


class Case:
    """Tokens given as (request, position) pairs over requests that hold `lens` entries; entries and pages that no token
    sees are rubbish (codes and values of NaN), pages of none of them -1."""

    def __init__(self, seed, tokens, lens, H, window, first, block, width=584, sink=False, skip=(), rubbish=True):
        rng = np.random.default_rng(seed)
        self.tokens, self.H, self.window, self.first, self.block = tokens, H, window, first, block
        self.skip = set(skip)
        need = [sref.cdiv(n, block) for n in lens]
        total = sum(need) + 2
        self.cache = sref.make_cache(rng, total, block, width)
        self.table = sref.make_tables(rng, lens, block, total)
        self.most = self.table.shape[1] * block
        looked = [set() for _ in lens]
        for t, (r, p) in enumerate(tokens):
            if t not in self.skip:
                looked[r].update(ref.seen(p, window, first, self.most))
        if rubbish:
            flat = self.cache.reshape(total, -1)
            for r, n in enumerate(lens):
                for b in range(need[r]):
                    if not any(j in looked[r] for j in range(b * block, (b + 1) * block)):
                        flat[self.table[r, b]] = 0xff
                        self.table[r, b] = -1
                for j in range(n):
                    page = self.table[r, j // block]
                    if j not in looked[r] and page >= 0:
                        flat[page, (j % block) * 576:(j % block + 1) * 576] = 0xff
        self.q = torch.from_numpy(2 * rng.standard_normal((len(tokens), H, 512))).bfloat16()
        self.sink = torch.from_numpy(rng.standard_normal(H)).float() if sink else None
        self.scale = 512 ** -0.5
        self.req = np.array([r for r, _ in tokens], np.int32)
        self.pos = np.array([p for _, p in tokens], np.int64)
        self.slots = np.array([-1 if t in self.skip else 5 for t in range(len(tokens))], np.int64)
        self.keys = {}

    def run(self, out_kind=torch.bfloat16, out=None, lse=None, stream=None, q=None):
        dev = [torch.from_numpy(a).cuda() for a in (self.cache, self.table, self.req, self.pos, self.slots)]
        T = len(self.tokens)
        out = torch.full((T, self.H, 512), 3.0, dtype=out_kind, device="cuda") if out is None else out
        lse = torch.full((T, self.H), 7.0, device="cuda") if lse is None else lse
        binding.window_attention(self.q.cuda() if q is None else q, dev[0], self.block, *dev[1:], self.window, self.scale, out,
                                 first=self.first, lse=lse, sink=None if self.sink is None else self.sink.cuda(), stream=stream)
        return out, lse

    def check(self, out, lse, tokens=None):
        half = sref.HALF_BF16 if out.dtype == torch.bfloat16 else sref.HALF_F32
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        sink = None if self.sink is None else self.sink.double().numpy()
        for t in range(len(self.tokens)) if tokens is None else tokens:
            r, p = self.tokens[t]
            if t in self.skip:
                assert (out[t] == 3).all() and (lse[t] == 7).all(), t
                continue
            at = ref.seen(p, self.window, self.first, self.most)
            for j in at:
                if (r, j) not in self.keys:
                    self.keys[r, j] = self.entry(self.table[r, j // self.block], j % self.block)
            k = np.stack([self.keys[r, j] for j in at]) if at else np.zeros((0, 512))
            k = k[~np.isnan(k).any(1)]  # (pages that are not there)
            want, l, tol, ltol = sref.attention(self.q[t].double().numpy(), k, self.scale, sink, half)
            # fp32 has no weight below 2^-126, and neither type a result: each such is 0, off by less than 2^-126 of its entry
            tol = tol + 2.0 ** -126 * (1 + np.abs(k).sum(0))
            assert (np.abs(out[t] - want) <= tol).all(), (t, np.max(np.abs(out[t] - want) / np.maximum(tol, 1e-300)))
            fine = np.isfinite(l)
            assert (np.abs(lse[t] - l)[fine] <= ltol[fine]).all() and (lse[t][~fine] == l[~fine]).all(), t

    def entry(self, page, off):
        if not 0 <= page < len(self.cache):
            return np.full(512, np.nan)
        return sref.entries(self.cache[page:page + 1], self.block, [0], off + 1)[off]


def consecutive(r, begin, n):
    return [(r, p) for p in range(begin, begin + n)]


CASES = {
    "one_token": dict(tokens=[(0, 0)], lens=[1], H=1, window=1, first=0, block=1),
    "window_of_one": dict(tokens=consecutive(0, 0, 70), lens=[70], H=3, window=1, first=2, block=2),
    "decode": dict(tokens=[(0, 999), (1, 4), (2, 127), (3, 128), (4, 131), (5, 132), (6, 500)], lens=[1000, 5, 128, 129, 132, 133, 501],
                   H=64, window=128, first=4, block=64, sink=True, skip=[6]),
    "decode_all_heads": dict(tokens=[(0, 300), (1, 77)], lens=[301, 78], H=128, window=128, first=0, block=16),
    "prefill": dict(tokens=consecutive(0, 0, 200) + consecutive(1, 333, 71), lens=[200, 404], H=64, window=128, first=4, block=64, sink=True),
    "prefill_odd": dict(tokens=consecutive(1, 7, 150), lens=[3, 157], H=33, window=100, first=0, block=67, width=592),
    "few_heads": dict(tokens=consecutive(0, 5, 133) + consecutive(1, 0, 40) + [(2, 9)], lens=[138, 40, 10], H=5, window=128, first=16,
                      block=3),
    "one_head": dict(tokens=consecutive(0, 0, 260), lens=[260], H=1, window=128, first=4, block=2),
    "sixteen_heads": dict(tokens=consecutive(0, 100, 37) + consecutive(1, 400, 5), lens=[137, 405], H=16, window=131, first=3, block=16),
    "small_window": dict(tokens=consecutive(0, 0, 90), lens=[90], H=20, window=7, first=3, block=4),
    "long_window": dict(tokens=consecutive(0, 1500, 9) + [(1, 900), (2, 3)], lens=[1509, 901, 4], H=16, window=1000, first=5, block=16),
    "window_past_all": dict(tokens=consecutive(0, 290, 10), lens=[300], H=40, window=(1 << 31) - 1, first=(1 << 31) - 1, block=64),
    "first_past_all": dict(tokens=consecutive(0, 290, 10), lens=[300], H=7, window=3, first=1000, block=64),
    "any_order": dict(tokens=[(1, 8), (0, 50), (0, 49), (1, 9), (1, 9), (0, 51), (0, 10), (2, 0), (1, 10), (0, 11)], lens=[52, 11, 1], H=8,
                      window=20, first=2, block=8),
    "skipped_between": dict(tokens=consecutive(0, 30, 40), lens=[70], H=12, window=33, first=1, block=8, skip=[0, 7, 8, 20, 39]),
}


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("name", CASES)
def test_window(name, kind):
    c = Case(len(name), **CASES[name])
    c.check(*c.run(kind))
    assert binding.device_errors() == 0


@pytest.mark.parametrize("window", [128, 200], ids=["short", "long"])
def test_positions_tables_and_requests_that_do_not_fit(window):
    tokens = [(0, 150), (1, 70), (2, 3), (0, 64), (3, 10), (1, 71)]
    c = Case(3, tokens, [130, 64, 4, 11], 24, window, 4, 64, sink=True, rubbish=False)
    if window == 128:
        c.table, c.most = c.table[:, :1].copy(), 64
    c.req[4] = -2
    c.skip.add(4)
    c.table[2, 0] = c.cache.shape[0]  # outside
    out, lse = c.run()
    assert binding.device_errors() == (2 if window == 128 else 4) | 4 | 1
    c.check(out, lse)


def test_nothing_to_see():
    """A table without columns, and a position whose entries are all left out: zeros, and an lse of the sink."""
    for sink in (False, True):
        c = Case(4, [(0, 5), (0, 300)], [64], 9, 20, 2, 64, sink=sink, rubbish=False)
        c.table[:] = -1
        out, lse = c.run()
        binding.device_errors()
        assert (out == 0).all()
        if sink:  # kept times log2(e) and given times log(2): two rounded constants, two products, half a step each
            assert ((lse - c.sink.cuda()).abs() <= 2.0 ** -22 * c.sink.cuda().abs()).all()
        else:
            assert (lse == -np.inf).all()
        c.table = c.table[:, :0]
        out, lse = c.run()
        assert binding.device_errors() == 2
        assert (out == 0).all()


@pytest.mark.parametrize("window,H", [(128, 64), (128, 6), (1000, 16)])
def test_strides(window, H):
    c = Case(8, consecutive(0, 40, 45), [85], H, window, 4, 8)
    whole_q = torch.zeros(H, 50, 520, dtype=torch.bfloat16, device="cuda")
    q = whole_q[:, 3:48, 8:].transpose(0, 1).copy_(c.q)
    out = torch.full((45, H + 1, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, 45), 7.0, device="cuda")
    c.run(out=out[:, 1:, :512], lse=lse.t(), q=q)
    c.check(out[:, 1:, :512], lse.t())
    assert (out[:, 0] == 3).all() and (out[:, :, 512:] == 3).all()


@pytest.mark.parametrize("window,first", [(128, 4), (2000, 0)])
def test_scores_of_any_size(window, first):
    """Scores far above and below 0, and entries of large magnitude, as the decode attention takes them."""
    for factor in (30.0, 1e-3, 2000.0):
        c = Case(21, consecutive(0, 100, 12), [112], 16, window, first, 16)
        c.q = (c.q.float() * factor).bfloat16()
        c.check(*c.run())
    c = Case(22, consecutive(0, 100, 12), [112], 16, window, first, 16, rubbish=False)
    scales = c.cache.reshape(c.cache.shape[0], -1)[:, 16 * 576:16 * 584]
    scales[:] = np.where(scales > 0, scales + 60, 0).astype(np.uint8)
    c.scale = 2.0 ** -60 * c.scale
    c.check(*c.run())


def test_same_as_decode_attention():
    """With a window past all entries and a token per request it is c128_decode_attention."""
    lens = [700, 64, 1, 129]
    c = Case(30, [(r, n - 1) for r, n in enumerate(lens)], lens, 32, 100000, 0, 16)
    out, lse = c.run()
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    binding.decode_attention(c.q.cuda(), torch.from_numpy(c.cache).cuda(), 16, torch.from_numpy(c.table).cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), c.scale, out2, lse=lse2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window", [128, 700])
def test_far_positions_and_many_tokens(window):
    """Positions near a million in blocks of 64, most of the table's blocks not held any more; a thousand tokens."""
    n, at = 1000, (1 << 20) - 1100
    rng = np.random.default_rng(5)
    H, block = 4, 64
    table = np.full((2, (1 << 20) // block), -1, np.int32)
    held = list(range((at - window) // block, (at + n) // block + 1)) + [0]
    table[1, held] = rng.permutation(len(held))
    cache = sref.make_cache(rng, len(held), block)
    tokens = consecutive(1, at, n)
    c = Case(1, [(0, 0)], [1], H, window, 4, block)
    c.tokens, c.cache, c.table, c.most = tokens, cache, table, 1 << 20
    c.q = torch.from_numpy(2 * rng.standard_normal((n, H, 512))).bfloat16()
    c.req, c.pos, c.slots = np.ones(n, np.int32), np.arange(at, at + n), np.zeros(n, np.int64)
    out, lse = c.run()
    assert binding.device_errors() == 0
    c.check(out, lse, tokens=[0, 1, 500, 777, 998, 999])


@pytest.mark.parametrize("window", [128, 700])
def test_graph_and_other_stream(window):
    c = Case(12, consecutive(0, 60, 50) + [(1, 20)], [110, 21], 18, window, 4, 16, sink=True)
    want = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    binding.reserve_workspace(1, s)
    dev = [torch.from_numpy(a).cuda() for a in (c.cache, c.table, c.req, c.pos, c.slots)]
    q, sink = c.q.cuda(), c.sink.cuda()
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.empty(binding.decode_attention_workspace(c.H), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(2):
                binding.window_attention(q, dev[0], c.block, *dev[1:], c.window, c.scale, out, first=c.first, lse=lse, sink=sink,
                                         workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    binding.release_stream(s)


@pytest.mark.parametrize("H", [64, 16, 5])
def test_entries_that_are_not_finite(H):
    """An entry with NaN makes the tokens that see it NaN, and no other: not those beside it in one item, nor those that
    come when it has left the window. The same for infinities. (Codes, rope values, and products without room.)"""
    tokens = consecutive(0, 0, 60) + consecutive(1, 0, 40)
    c = Case(40, tokens, [60, 40], H, 12, 2, 8, rubbish=False)
    flat = c.cache.reshape(c.cache.shape[0], -1)

    def entry(r, j):
        page, off = c.table[r, j // 8], j % 8
        return flat[page, off * 576:off * 576 + 576], flat[page, 8 * 576 + off * 8:8 * 576 + off * 8 + 8]

    entry(0, 20)[0][100] = 0xff
    entry(0, 41)[0][448:].view(np.uint16)[5] = 0x7f80
    entry(1, 1)[0][448:].view(np.uint16)[63] = 0xffc0   # one of the first entries: seen to the end
    entry(1, 0)[1][3] = 255
    out, lse = c.run()
    bad = [any((r, j) in ((0, 20), (0, 41), (1, 1), (1, 0)) for j in ref.seen(p, 12, 2, 1 << 20)) for r, p in tokens]
    bad = torch.tensor(bad, device="cuda")
    assert 0 < bad.sum() < len(tokens)
    assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    c.check(out, lse, tokens=[t for t in range(len(tokens)) if not bad[t]])


def test_rows_that_are_not_finite():
    """A query with NaN makes its own row NaN, and no other."""
    c = Case(41, consecutive(0, 50, 20), [70], 16, 12, 2, 8)
    c.q[3, 5, 100] = float("nan")
    c.q[9, 0, 500] = float("inf")
    out, lse = c.run()
    torch.cuda.synchronize()
    assert torch.isnan(out[3, 5]).all() and torch.isnan(lse[3, 5])
    c.q[3, 5, 100] = c.q[9, 0, 500] = 0
    keep = [t for t in range(20) if t not in (3, 9)]
    c.check(out, lse, tokens=keep)
    other = [h for h in range(16) if h != 5]
    ref_out, ref_lse = c.run()
    assert torch.equal(out[3, other], ref_out[3, other]) and torch.equal(out[9, 1:], ref_out[9, 1:])


@pytest.mark.parametrize("H", [64, 16])
def test_entries_of_any_magnitude_that_are_not_seen(H):
    """Entries so large that a score with them has no room, beside tokens that do not see them."""
    c = Case(42, consecutive(0, 0, 60), [60], H, 12, 2, 8, rubbish=False)
    flat = c.cache.reshape(c.cache.shape[0], -1)
    for j in (20, 33):
        page, off = c.table[0, j // 8], j % 8
        flat[page, 8 * 576 + off * 8:8 * 576 + off * 8 + 7] = 246  # 2^119
        flat[page, off * 576:off * 576 + 448] = 0x7e               # 448
    c.q[:] = c.q.abs()
    out, lse = c.run()
    c.check(out, lse, tokens=[t for t in range(60) if not (20 <= t < 32 or 33 <= t < 45)])


@pytest.mark.parametrize("window,first", [(128, 4), (700, 4), (136, 0), (1, 135)])
def test_the_last_positions_of_32_bits(window, first):
    """A table of 2^31 - 1 entries, positions up to its end, behind it, and the largest of 64 bits."""
    most, block, n = (1 << 31) - 1, 64, 70
    rng = np.random.default_rng(6)
    table = np.full((1, 1 << 25), -1, np.int32)
    held = list(range(first // block + 1)) + list(range((most - n - window) // block, 1 << 25))
    table[0, held] = rng.permutation(len(held))
    tokens = consecutive(0, most - n, n + 2) + [(0, most + 100), (0, (1 << 63) - 1)]
    c = Case(1, [(0, 0)], [1], 5, window, first, block)
    c.tokens, c.table, c.most = tokens, table, most
    c.cache = sref.make_cache(rng, len(held), block)
    T = len(tokens)
    c.q = torch.from_numpy(2 * rng.standard_normal((T, 5, 512))).bfloat16()
    c.req, c.pos, c.slots = np.zeros(T, np.int32), np.array([p for _, p in tokens]), np.zeros(T, np.int64)
    out, lse = c.run()
    assert binding.device_errors() == 2  # a position behind the table
    c.check(out, lse)


def drafts(begins, counts):
    """Some consecutive tokens of each request."""
    return [(r, p) for r, (b, n) in enumerate(zip(begins, counts)) for p in range(b, b + n)]


# Long windows of few heads, where tokens that follow one another are taken together. (That is done where there is work enough
# for the whole GPU and three tokens to a row of the table, so one more request has a long prompt.)
RUNS = {
    "four_each": dict(tokens=drafts([1000, 3, 700, 150, 0, 436], [4] * 6), lens=[1004, 7, 704, 154, 4, 440], H=16, window=300, first=4, block=16),
    "no_first": dict(tokens=drafts([2000, 511], [4, 4]), lens=[2004, 515], H=16, window=1024, first=0, block=64, sink=True),
    "uneven": dict(tokens=drafts([90, 801, 402, 300, 222, 10], [3, 1, 5, 9, 2, 6]), lens=[93, 802, 407, 309, 224, 16], H=13, window=201, first=3,
                   block=2, sink=True),
    "wide_blocks": dict(tokens=drafts([600, 601, 60], [7, 8, 8]), lens=[607, 609, 68], H=12, window=333, first=0, block=67, width=592),
    "many_first": dict(tokens=drafts([600, 199, 250], [7, 8, 4]), lens=[607, 207, 254], H=5, window=137, first=200, block=16),
    "one_head": dict(tokens=drafts([100, 900], [40, 41]), lens=[140, 941], H=1, window=450, first=1, block=64),
    "skipped": dict(tokens=drafts([500, 700], [12, 12]), lens=[512, 712], H=16, window=190, first=2, block=8, skip=[0, 5, 6, 11, 12, 23]),
    "apart": dict(tokens=[(r, 300 + 7 * r) for r in range(12)] + drafts([50], [8]), lens=[301 + 7 * r for r in range(12)], H=16, window=160,
                  first=4, block=16),
    "one_long": dict(tokens=drafts([5000], [4]), lens=[5004], H=8, window=4096, first=4, block=16, sink=True),
    "twice": dict(tokens=drafts([400], [4]) + drafts([400], [4]) + [(0, 402)] * 3, lens=[404], H=16, window=150, first=0, block=16),
}


def with_a_prompt(tokens, lens, window, first, **rest):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = -(-9 * sms // (min(window + first, max(lens)) // 64 + 1))
    return dict(tokens=tokens + consecutive(len(lens), 0, n), lens=lens + [n], window=window, first=first, **rest)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("name", RUNS)
def test_runs_of_tokens(name, kind):
    c = Case(len(name) + 100, **with_a_prompt(**RUNS[name]))
    n = len(RUNS[name]["tokens"])
    c.check(*c.run(kind), tokens=[*range(n), *range(n, len(c.tokens), 19)])
    assert binding.device_errors() == 0


@pytest.mark.parametrize("H", [16, 3])
def test_runs_with_entries_that_are_not_finite(H):
    """Entries that some tokens of a run see and others do not: at either end of the window, and the tokens' own."""
    tokens = drafts([400, 300, 500], [8, 8, 8])
    c = Case(43, **with_a_prompt(tokens, [408, 308, 508], 200, 2, H=H, block=8, rubbish=False))
    flat = c.cache.reshape(c.cache.shape[0], -1)

    def entry(r, j):
        page, off = c.table[r, j // 8], j % 8
        return flat[page, off * 576:off * 576 + 576], flat[page, 8 * 576 + off * 8:8 * 576 + off * 8 + 8]

    bad_entries = [(0, 403), (1, 102), (2, 504), (2, 303)]
    entry(0, 403)[0][100] = 0xff
    entry(1, 102)[0][448:].view(np.uint16)[5] = 0x7f80
    entry(2, 504)[1][3] = 255
    entry(2, 303)[0][448:].view(np.uint16)[63] = 0xffc0
    out, lse = c.run()
    bad = torch.tensor([any((r, j) in bad_entries for j in ref.seen(p, 200, 2, 1 << 20)) for r, p in tokens], device="cuda")
    assert 0 < bad.sum() < len(tokens)
    assert torch.isnan(out[:24][bad].float()).all() and torch.isnan(lse[:24][bad]).all()
    c.check(out, lse, tokens=[t for t in range(len(tokens)) if not bad[t]] + [30, 99, len(c.tokens) - 1])


@pytest.mark.parametrize("factor", [1.0, 30.0, -2000.0])
def test_runs_whose_first_entries_are_not_there(factor):
    """Pages that are not there, so that of a run's first tile the last token sees nothing, and the first tokens an entry each."""
    tokens = drafts([500, 800], [4, 4])
    c = Case(44, **with_a_prompt(tokens, [504, 804], 200, 0, H=16, block=1, rubbish=False))
    c.q = (c.q.float() * factor).bfloat16()
    c.table[0, 304:430] = -1
    c.table[1, 601:660] = c.cache.shape[0] + 5
    out, lse = c.run()
    assert binding.device_errors() == 4
    c.check(out, lse, tokens=range(30))


@pytest.mark.parametrize("H", [16, 7])
def test_runs_and_large_entries_that_are_not_seen(H):
    """Entries so large that a score with them has no room, seen by some tokens of a run: the others are not touched."""
    tokens = drafts([400, 600], [8, 8])
    c = Case(45, **with_a_prompt(tokens, [408, 608], 180, 2, H=H, block=8, rubbish=False))
    flat = c.cache.reshape(c.cache.shape[0], -1)
    large = [(0, 402), (0, 226), (1, 605), (1, 422)]
    for r, j in large:
        page, off = c.table[r, j // 8], j % 8
        flat[page, 8 * 576 + off * 8:8 * 576 + off * 8 + 7] = 246  # 2^119
        flat[page, off * 576:off * 576 + 448] = 0x7e               # 448
    c.q[:] = c.q.abs()
    out, lse = c.run()
    c.check(out, lse, tokens=[t for t, (r, p) in enumerate(tokens) if not any((r, j) in large for j in ref.seen(p, 180, 2, 1 << 20))])


def test_runs_with_strides_from_a_graph_and_scores_of_any_size():
    tokens = drafts([400, 600, 17], [8, 7, 9])
    for factor in (1.0, 40.0):
        c = Case(46, **with_a_prompt(tokens, [408, 607, 26], 180, 2, H=10, block=16, sink=True))
        c.q = (c.q.float() * factor).bfloat16()
        T = len(c.tokens)
        q = torch.zeros(10, T + 4, 520, dtype=torch.bfloat16, device="cuda")[:, 3:T + 3, 8:].transpose(0, 1).copy_(c.q)
        out = torch.full((T, 11, 520), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((10, T), 7.0, device="cuda")
        c.run(out=out[:, 1:, :512], lse=lse.t(), q=q)
        c.check(out[:, 1:, :512], lse.t(), tokens=[*range(24), *range(24, T, 29)])
        assert (out[:, 0] == 3).all() and (out[:, :, 512:] == 3).all()
        dev = [torch.from_numpy(a).cuda() for a in (c.cache, c.table, c.req, c.pos, c.slots)]
        out2, sink = torch.zeros(T, 10, 512, dtype=torch.bfloat16, device="cuda"), c.sink.cuda()
        ws = torch.empty(binding.decode_attention_workspace(10), dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        binding.reserve_workspace(1, s)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                binding.window_attention(q, dev[0], c.block, *dev[1:], c.window, c.scale, out2, first=c.first, sink=sink, workspace=ws)
        for _ in range(2):
            ws.fill_(255)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out2, out[:, 1:, :512])
        binding.release_stream(s)


@pytest.mark.parametrize("H", [64, 16, 3])
def test_a_decode_batch_padded_at_its_end(H):
    """More tokens than CTAs, less than two to a request: dealt out in turn."""
    rng = np.random.default_rng(60)
    lens = [int(n) for n in rng.integers(1, 300, 330)]
    tokens = [(r, n - 1) for r, n in enumerate(lens)] + [(5, lens[5] - 1), (5, max(0, lens[5] - 2))] + [(0, 0)] * 180
    c = Case(61, tokens, lens, H, 40, 3, 1, sink=True, skip=[0, 17, *range(332, 512)])
    c.check(*c.run())
    assert binding.device_errors() == 0


def test_runs_with_queries_that_are_not_finite():
    """A query with NaN or infinity, in a run: its own row, and no other."""
    tokens = drafts([400, 600], [8, 8])
    c = Case(47, **with_a_prompt(tokens, [408, 608], 180, 2, H=9, block=8))
    clean = c.run()
    c.check(*clean, tokens=range(16))
    c.q[2, 5, 100] = float("nan")
    c.q[13, 0, 500] = float("inf")
    out, lse = c.run()
    torch.cuda.synchronize()
    assert torch.isnan(out[2, 5]).all() and torch.isnan(lse[2, 5])
    c.q[2, 5, 100] = c.q[13, 0, 500] = 0
    c.check(out, lse, tokens=[t for t in range(16) if t not in (2, 13)])
    rest = [h for h in range(9) if h != 5]
    # (other rows of the two tokens: weights relative to other references, so not bit for bit)
    assert not torch.isnan(out[2, rest]).any() and not torch.isnan(out[13, 1:]).any()


def test_runs_past_the_table_and_of_requests_that_do_not_fit():
    tokens = drafts([500, 700, 300], [8, 8, 8])
    c = Case(48, **with_a_prompt(tokens, [508, 708, 308], 190, 3, H=16, block=4, rubbish=False))
    c.table, c.most = c.table[:, :176].copy(), 704   # the second request's tokens pass 704 within a run
    c.req[[16, 21]] = -1, len(c.table)
    c.skip.update((16, 21))
    c.slots[18] = -1
    c.skip.add(18)
    out, lse = c.run()
    assert binding.device_errors() == 2 | 1
    c.check(out, lse, tokens=[*range(24), 30, 99])


def test_a_run_over_many_tokens_in_every_place_of_four():
    """Requests of one to nine tokens, so that runs begin and end in every place, with skipped rows between."""
    rng = np.random.default_rng(62)
    counts = [int(n) for n in rng.integers(1, 10, 90)]
    begins = [int(n) for n in rng.integers(0, 400, 90)]
    tokens = drafts(begins, counts)
    skip = sorted(rng.choice(len(tokens), 40, replace=False).tolist())
    c = Case(63, tokens, [b + n for b, n in zip(begins, counts)], 7, 230, 5, 1, sink=True, skip=skip)
    c.check(*c.run())
    assert binding.device_errors() == 0
