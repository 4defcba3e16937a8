"""c128_decode_attention and c128_merge_attention against plain attention in 64 bits. The tolerances are derived in
serving_ref.attention (sums in fp32, weights and results rounded to bf16) and beside the merge."""
import numpy as np
import pytest

from serving_ref import (HALF_BF16, HALF_F32, HEAD, NOPE, RECORD, attention, cdiv, e4m3_values, entries, make_cache,
                         make_tables, merge)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def binding():
    from deepseek_v4_sparse_c128_gb300 import binding as b
    from deepseek_v4_sparse_c128_gb300 import build
    build.build()
    b.load()
    b.device_errors(clear=True)
    return b


def _cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _queries(rng, R, H, size=2.0):
    import torch
    return torch.from_numpy((size * rng.standard_normal((R, H, HEAD))).astype(np.float32)).to(torch.bfloat16).cuda()


def _case(rng, lens, H, block, width=584, spare=2, size=2.0, sink=False):
    need = sum(cdiv(max(0, int(n)), block) for n in lens)
    cache = make_cache(rng, need + spare, block, width)
    return {"q": _queries(rng, len(lens), H, size), "cache": cache, "block": block, "lens": np.array(lens, np.int32),
            "table": make_tables(rng, lens, block, need + spare), "scale": HEAD ** -0.5,
            "sink": rng.standard_normal(H).astype(np.float32) if sink else None}


def _run(binding, c, out=None, lse=None, expect_bits=0, **kw):
    import torch
    R, H = c["q"].shape[:2]
    out = torch.full((R, H, HEAD), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((R, H), 7.0, device="cuda") if lse is None else lse
    binding.decode_attention(c["q"], c.get("cache_gpu", None) if "cache_gpu" in c else _cuda(c["cache"]), c["block"],
                             _cuda(c["table"]), _cuda(c["lens"]), c["scale"], out, lse=lse,
                             sink=None if c["sink"] is None else _cuda(c["sink"]), **kw)
    assert binding.device_errors(clear=True) == expect_bits
    return out, lse


def _check(c, out, lse, requests=None, out_half=HALF_BF16):
    """Every given request's result against 64 bits; entries of pages outside the cache are left out."""
    out, lse, q = out.double().cpu().numpy(), lse.double().cpu().numpy(), c["q"].double().cpu().numpy()
    for r in range(len(c["lens"])) if requests is None else requests:
        n = min(max(0, int(c["lens"][r])), c["table"].shape[1] * c["block"])
        k = entries(c["cache"], c["block"], c["table"][r], n)
        pages = c["table"][r][np.arange(n) // c["block"]] if n else np.zeros(0)
        k = k[(pages >= 0) & (pages < c["cache"].shape[0])]
        want, want_lse, tol, tol_lse = attention(q[r], k, c["scale"], c["sink"], out_half)
        assert np.array_equal(np.isneginf(want_lse), np.isneginf(lse[r])), r
        real = np.isfinite(want_lse)
        assert np.array_equal(np.isfinite(want_lse), np.isfinite(lse[r])), r
        assert (np.abs(lse[r] - want_lse)[real] <= tol_lse[real]).all(), (r, np.abs(lse[r] - want_lse)[real].max())
        off = np.abs(out[r] - want) - tol
        assert (off <= 0).all(), (r, n, np.unravel_index(off.argmax(), off.shape), off.max())


LENS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 200, 0, 301]


@pytest.mark.parametrize("block", [1, 2, 64, 67])
@pytest.mark.parametrize("heads", [1, 16, 33, 64])
def test_decode_lengths_and_blocks(binding, heads, block):
    rng = np.random.default_rng([heads, block])
    c = _case(rng, LENS, heads, block, sink=heads % 2 == 1)
    out, lse = _run(binding, c)
    _check(c, out, lse)


@pytest.mark.parametrize("heads", [2, 15, 17, 31, 48, 63, 65, 128, 130, 200, 1000, 1024])
def test_decode_heads(binding, heads):
    rng = np.random.default_rng(heads)
    c = _case(rng, [70, 3, 0, 150], heads, 16, sink=heads % 2 == 0)
    out, lse = _run(binding, c)
    _check(c, out, lse)


@pytest.mark.parametrize("requests,heads,longest", [(1, 64, 5000), (1, 8, 20000), (3, 128, 2000), (2, 16, 1), (1, 1, 64),
                                                    (1, 128, 129), (40, 4, 700), (170, 20, 130), (700, 3, 90),
                                                    (9000, 3, 2)])
def test_decode_split_over_the_cache(binding, requests, heads, longest):
    """Requests split over many CTAs, and many requests to a CTA."""
    rng = np.random.default_rng([requests, heads, longest])
    lens = rng.integers(0, longest + 1, requests)
    lens[0] = longest
    c = _case(rng, lens, heads, 64 if longest > 1000 else 7)
    out, lse = _run(binding, c)
    _check(c, out, lse, None if requests < 50 else list(range(0, requests, 7 if requests < 1000 else 90)))


def test_decode_is_deterministic(binding):
    rng = np.random.default_rng(11)
    c = _case(rng, [3000, 10, 777], 64, 64)
    first = _run(binding, c)
    for _ in range(3):
        again = _run(binding, c)
        assert (first[0].view(dtype=__import__("torch").int16) == again[0].view(dtype=__import__("torch").int16)).all()
        assert (first[1] == again[1]).all()


def test_decode_strides_and_types(binding):
    """Heads before requests, padded rows, a padded cache and table, fp32 results, no lse."""
    import torch
    rng = np.random.default_rng(5)
    lens = [100, 0, 31, 65]
    c = _case(rng, lens, 24, 3, width=600)
    q = torch.full((24, 4, HEAD + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    q[:, :, :HEAD] = c["q"].transpose(0, 1)
    c["q"] = q[:, :, :HEAD].transpose(0, 1)
    table = np.full((4, c["table"].shape[1] + 5), -1, np.int32)
    table[:, :c["table"].shape[1]] = c["table"]
    c["table"] = table
    whole = torch.full((24, 4, HEAD + 16), 7.0, device="cuda")
    lse = torch.full((24, 4), 7.0, device="cuda")
    out = whole[:, :, :HEAD].transpose(0, 1)
    _run(binding, c, out=out, lse=lse.t())
    _check(c, out, lse.t(), out_half=HALF_F32)
    assert bool((whole[:, :, HEAD:] == 7).all())
    out = torch.empty(4, 24, HEAD, dtype=torch.bfloat16, device="cuda")
    binding.decode_attention(c["q"], _cuda(c["cache"]), 3, _cuda(table), _cuda(c["lens"]), c["scale"], out)
    _check(c, out, lse.t())
    assert binding.device_errors(clear=True) == 0


def test_decode_every_code_and_scale(binding):
    """With one entry the weight is 1 and the result is the entry itself, exactly."""
    values = e4m3_values()
    block = 4
    scale_bytes = list(range(8, 247, 2)) + [127, 134, 135, 136]
    cache = np.zeros((len(scale_bytes), block, 584), np.uint8)
    codes = np.array([b for b in range(256) if b & 127 != 127] + [0, 0], np.uint8)
    for i, sb in enumerate(scale_bytes):
        flat, off = cache[i].reshape(-1), i % block
        flat[off * RECORD:off * RECORD + NOPE] = np.resize(np.roll(codes, 64 * (i % 4)), NOPE)
        flat[block * RECORD + off * 8:][:7] = sb
        flat[off * RECORD + NOPE:off * RECORD + RECORD] = np.arange(64, dtype=np.uint16).view(np.uint8) if i % 2 else 0x3f
    # entry i sits at offset i % block of page i: a request of 1 entry reads offset 0, so shift the records there
    for i in range(len(scale_bytes)):
        flat, off = cache[i].reshape(-1), i % block
        rec, sc = flat[off * RECORD:(off + 1) * RECORD].copy(), flat[block * RECORD + off * 8:][:8].copy()
        flat[:RECORD] = rec
        flat[block * RECORD:][:8] = sc
    R = len(scale_bytes)
    import torch
    c = {"q": torch.zeros(R, 5, HEAD, dtype=torch.bfloat16, device="cuda"), "cache": cache, "block": block,
         "lens": np.ones(R, np.int32), "table": np.arange(R, dtype=np.int32)[:, None], "scale": 1.0, "sink": None}
    out, lse = _run(binding, c)
    for r in range(R):
        want = entries(cache, block, c["table"][r], 1)[0]
        with np.errstate(over="ignore"):
            got = out[r].double().cpu().numpy()
        real = np.abs(want) < 2.0 ** 127
        assert np.array_equal(got[:, real], np.broadcast_to(want[real], (5, int(real.sum())))), scale_bytes[r]
    assert bool((lse == 0).all())
    assert values[127] != values[127]


def test_decode_infinities_and_nan(binding):
    """NaN codes in an entry reach every head of that request, a NaN query its own head; stale bytes reach nobody."""
    import torch
    rng = np.random.default_rng(8)
    lens = [70, 70, 70, 5]
    c = _case(rng, lens, 8, 16)
    cache = c["cache"]
    cache[c["table"][0, 1]].reshape(-1)[3 * RECORD + 100] = 0x7f            # entry 19 of request 0, column 100
    stale = cache[c["table"][2, 4]].reshape(-1)                             # entries 64..79 of request 2: 6 real
    stale[6 * RECORD:16 * RECORD] = 0xff
    stale[16 * RECORD + 6 * 8:16 * RECORD + 16 * 8] = 0xff
    c["q"][1, 3, 17] = float("nan")
    c["q"][3, 2, 500] = float("inf")
    out, lse = _run(binding, c)
    assert bool(out[0].isnan().any(-1).all()) and bool(lse[0].isnan().all())
    assert bool(out[1, 3].isnan().all()) and bool(lse[1, 3].isnan())
    assert bool(out[3, 2].isnan().any()) and not bool(out[3, :2].isnan().any()) and not bool(out[3, 3:].isnan().any())
    keep = [0, 1, 2, 4, 5, 6, 7]
    one = dict(c, q=c["q"][:, keep].contiguous())
    _check(one, out[:, keep], lse[:, keep], [1])
    _check(c, out, lse, [2])


def test_decode_bad_pages_and_lengths(binding):
    rng = np.random.default_rng(9)
    lens = [100, 40, 200, 64, 33]
    c = _case(rng, lens, 20, 8, sink=True)
    c["table"][0, 3] = -1
    c["table"][0, 12] = c["cache"].shape[0]
    c["table"][3, :8] = -5                          # nothing left of request 3
    c["table"][2, 24] = 2147483647
    out, lse = _run(binding, c, expect_bits=4)
    _check(c, out, lse)
    c["lens"] = np.array([100, -7, c["table"].shape[1] * 8 + 1, 0, 2147483647], np.int32)
    c["table"][:] = rng.integers(0, c["cache"].shape[0], c["table"].shape)
    out, lse = _run(binding, c, expect_bits=2 | 128)
    _check(c, out, lse)


@pytest.mark.parametrize("heads", [5, 32, 100])
@pytest.mark.parametrize("sink", [False, True])
def test_decode_of_one_entry_is_that_entry(binding, heads, sink):
    """The weights' rounding cancels: with one entry the result is the entry, to the bit, and without rounding in lse;
    with a sink it is the entry times its share, rounded once."""
    rng = np.random.default_rng([18, heads])
    c = _case(rng, [1] * 40, heads, 64, size=4.0, sink=sink)
    out, lse = _run(binding, c)
    out, lse, q = out.double().cpu().numpy(), lse.double().cpu().numpy(), c["q"].double().cpu().numpy()
    for r in range(40):
        k = entries(c["cache"], 64, c["table"][r], 1)[0]
        s = c["scale"] * (q[r] @ k)
        if not sink:
            assert np.array_equal(out[r], np.broadcast_to(k, out[r].shape))
            # the score: 512 products in fp32, then log2 and back
            assert (np.abs(lse[r] - s) <= 600 * HALF_F32 * (c["scale"] * (np.abs(q[r]) @ np.abs(k)) + 1)).all()
        else:
            share = 1 / (1 + np.exp(c["sink"].astype(np.float64) - s))
            # half a step of bf16, and the score's error and three operations of 2^-22 in the share
            off = 600 * HALF_F32 * (c["scale"] * (np.abs(q[r]) @ np.abs(k)) + 1) + 2.0 ** -20
            want = share[:, None] * k[None]
            assert (np.abs(out[r] - want) <= np.abs(want) * (HALF_BF16 * (1 + 2.0 ** -8) + off[:, None])).all()


def test_decode_growing_scores(binding):
    """Scores that climb from tile to tile by far more than an exponential holds, and ones that fall."""
    import torch
    rng = np.random.default_rng(10)
    n = 900
    c = _case(rng, [n, n], 9, 64)
    for r, sign in ((0, 1), (1, -1)):
        for j in range(n):                          # rope column 0 of entry j: the query's only non-zero column
            rec = c["cache"][c["table"][r, j // 64]].reshape(-1)[(j % 64) * RECORD:][:RECORD]
            x = np.float32(sign * (j - n / 2) * 1.5)
            rec[NOPE:NOPE + 2] = np.array([x], np.float32).view(np.uint16)[1:].view(np.uint8)
    c["q"][:] = 0
    c["q"][:, :, NOPE] = torch.arange(9, device="cuda") / 2 - 1
    c["scale"] = 1.0
    out, lse = _run(binding, c)
    _check(c, out, lse)
    c["scale"] = -1.0
    out, lse = _run(binding, c)
    _check(c, out, lse)


@pytest.mark.parametrize("scale", [1e20, -1e20, 3e35, 1e-30])
def test_decode_huge_and_tiny_scores(binding, scale):
    """Scores whose steps in fp32 are wider than any reference's slack (all weight goes to the highest), and all equal."""
    import torch
    rng = np.random.default_rng(16)
    n = 400
    c = _case(rng, [n, 70], 17, 64)
    rank = rng.permutation(n)
    for r in range(2):
        for j in range(n if r == 0 else 70):        # entry j's rope column 0 holds rank[j] - 200, exact in bf16
            rec = c["cache"][c["table"][r, j // 64]].reshape(-1)[(j % 64) * RECORD:][:RECORD]
            x = np.array([np.float32(rank[j] - 200)]).view(np.uint32)[0]
            assert x & 0xffff == 0
            rec[NOPE:NOPE + 2] = np.array([x >> 16], np.uint16).view(np.uint8)
    c["q"][:] = 0
    c["q"][:, :, NOPE] = 1
    c["scale"] = scale
    out, lse = _run(binding, c)
    if abs(scale) < 1:
        _check(c, out, lse)
        return
    for r, m in ((0, n), (1, 70)):
        best = int(np.argmax(rank[:m]) if scale > 0 else np.argmin(rank[:m]))
        want = entries(c["cache"], 64, c["table"][r], m)[best]
        assert np.array_equal(out[r].double().cpu().numpy(), np.broadcast_to(want, (17, HEAD)))
        top = abs(scale) * abs(rank[best] - 200)
        assert np.allclose(lse[r].double().cpu().numpy(), top, rtol=2.0 ** -21, atol=0)


def test_decode_far_pages(binding):
    """A cache of more than 4 GiB whose used pages sit behind that."""
    import torch
    rng = np.random.default_rng(12)
    block, pages = 64, 120000                        # 4.5 GB
    small = _case(rng, [150, 64], 16, block)
    cache = torch.zeros(pages, block, 584, dtype=torch.uint8, device="cuda")
    far = pages - small["cache"].shape[0]
    cache[far:] = _cuda(small["cache"])
    c = dict(small, cache_gpu=cache, table=np.where(small["table"] >= 0, small["table"] + far, -1).astype(np.int32))
    out, lse = _run(binding, c)
    _check(small, out, lse)


def test_decode_graph_replays_with_other_lengths(binding):
    """Captured once, replayed while lengths and tables change; two graphs with a workspace each at the same time."""
    import torch
    rng = np.random.default_rng(13)
    c = _case(rng, [600, 640, 1000], 33, 64)
    cache, table, q = _cuda(c["cache"]), _cuda(c["table"]), c["q"]
    graphs = []
    for k in range(2):
        s = torch.cuda.Stream()
        lens, out, lse = _cuda(c["lens"]), torch.empty_like(q), torch.empty(3, 33, device="cuda")
        ws = torch.empty(binding.decode_attention_workspace(33), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        binding.reserve_workspace(1, stream=s)
        with torch.cuda.stream(s):
            op = binding.PreparedOp("decode_attention", q, cache, 64, table, lens, c["scale"], out, lse=lse, workspace=ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                op()
        graphs.append((s, g, lens, out, lse, op))
    for lengths in ([[600, 40, 1000], [0, 1, 65]], [[5, 640, 300], [600, 0, 999]]):
        for (s, g, lens, out, lse, _), want in zip(graphs, lengths):
            lens.copy_(_cuda(np.array(want, np.int32)))
        torch.cuda.synchronize()
        for s, g, *_ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (s, g, lens, out, lse, _), want in zip(graphs, lengths):
            assert binding.device_errors(s, clear=True) == 0
            _check(dict(c, lens=np.array(want, np.int32)), out, lse)


def test_decode_on_another_stream_behind_its_producer(binding):
    import torch
    rng = np.random.default_rng(14)
    c = _case(rng, [900, 77], 64, 64)
    s = torch.cuda.Stream()
    args = (_cuda(c["cache"]), 64, _cuda(c["table"]), _cuda(c["lens"]), c["scale"])
    out, q = torch.zeros_like(c["q"]), torch.zeros_like(c["q"])
    lse = torch.zeros(2, 64, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20000000)
        q.copy_(c["q"])
        binding.decode_attention(q, *args, out, lse=lse)
        got, got_lse = out.clone(), lse.clone()
        out.zero_()
    s.synchronize()
    assert binding.device_errors(s, clear=True) == 0
    _check(c, got, got_lse)


def test_decode_refuses_a_small_workspace(binding):
    import torch
    rng = np.random.default_rng(15)
    c = _case(rng, [10], 4, 8)
    ws = torch.empty(binding.decode_attention_workspace(4) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(binding.C128Error) as e:
        _run(binding, c, workspace=ws)
    assert e.value.status == 7


def test_decode_gives_up_after_a_wait_that_runs_out(binding):
    """CTA 0 never learns of its tiles: the call ends with the TIMEOUT bit, the other CTAs' requests are there, what
    CTA 0 had to store is as it was, and the next call is right."""
    import torch
    rng = np.random.default_rng(17)
    c = _case(rng, [64] * 400, 16, 64)               # one tile each, whole requests only
    args = (c["q"], _cuda(c["cache"]), 64, _cuda(c["table"]), _cuda(c["lens"]), c["scale"])
    out = torch.full((400, 16, HEAD), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((400, 16), 7.0, device="cuda")
    torch.cuda.synchronize()
    binding.debug_stall_decode_attention(*args, out, lse=lse)
    assert binding.device_errors(clear=True) == 32
    untouched = (out == 7).all(-1).all(-1)
    n = int(untouched.sum())
    assert 1 <= n <= 5 and bool(untouched[:n].all())  # the first column's run
    _check(c, out, lse, list(range(n, 400, 13)))
    out, lse = _run(binding, c)
    _check(c, out, lse, list(range(0, 400, 13)))


# ------------------------------------------------------------------------------------------ merge
@pytest.mark.parametrize("part_f32", [False, True])
@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("parts,requests,heads", [(1, 1, 1), (2, 3, 5), (4, 7, 64), (5, 2, 33), (9, 1, 8)])
def test_merge(binding, parts, requests, heads, part_f32, out_f32):
    import torch
    g = torch.Generator(device="cuda").manual_seed(parts * 100 + heads)
    part = torch.randn(parts, requests, heads, HEAD, generator=g, device="cuda")
    lse = 20 * torch.randn(parts, requests, heads, generator=g, device="cuda")
    gone = torch.rand(parts, requests, heads, generator=g, device="cuda") < 0.3
    lse[gone] = -float("inf")
    part[gone] = float("nan")                       # nothing there is used
    lse[:, 0, 0] = -float("inf")                    # a row that saw nothing at all
    part = part if part_f32 else part.to(torch.bfloat16)
    out = torch.full((requests, heads, HEAD), 7.0, dtype=torch.float32 if out_f32 else torch.bfloat16, device="cuda")
    out_lse = torch.full((heads, requests), 7.0, device="cuda")
    binding.merge_attention(part, lse, out, lse=out_lse.t())
    want, want_lse, mag = merge(part.double().cpu().numpy(), lse.double().cpu().numpy())
    # exp, the sums and the division in fp32: a few steps of 2^-24 each on the magnitudes, and exp of a difference d
    # of two fp32 values off by 2^-24 |d| more, |d| < 120: together below 2^-16; then one rounding of the result
    tol = (HALF_F32 if out_f32 else HALF_BF16) * np.abs(want) + 2.0 ** -16 * mag
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    got = out_lse.t().double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(want_lse)) and np.isneginf(got[0, 0])
    real = ~np.isneginf(want_lse)
    assert (np.abs(got - want_lse)[real] <= 2.0 ** -16 + 2.0 ** -22 * np.abs(want_lse[real])).all()


def test_merge_in_place_and_strided(binding):
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    part = torch.randn(6, 3, 40, 2 * HEAD, generator=g, device="cuda").to(torch.bfloat16)[:, :, :, :HEAD].transpose(1, 2)
    lse = torch.randn(40, 3, 6, generator=g, device="cuda").permute(2, 0, 1)
    want, want_lse, mag = merge(part.double().cpu().numpy(), lse.double().cpu().numpy())
    binding.merge_attention(part, lse, part[4], lse=lse[4])
    assert (np.abs(part[4].double().cpu().numpy() - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -16 * mag).all()
    assert (np.abs(lse[4].double().cpu().numpy() - want_lse) <= 2.0 ** -16).all()


def test_attention_in_two_parts_is_attention_over_all(binding):
    """A cache cut in two, attended to separately and merged, against attention over the whole."""
    import torch
    rng = np.random.default_rng(21)
    c = _case(rng, [500, 128, 64, 0], 40, 64)
    first = np.minimum(c["lens"], 128).astype(np.int32)
    rest = (c["lens"] - first).astype(np.int32)
    part = torch.empty(2, 4, 40, HEAD, device="cuda")
    lse = torch.empty(2, 4, 40, device="cuda")
    _run(binding, dict(c, lens=first), out=part[0], lse=lse[0])
    _run(binding, dict(c, lens=rest, table=np.ascontiguousarray(c["table"][:, 2:])), out=part[1], lse=lse[1])
    out, out_lse = torch.empty(4, 40, HEAD, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 40, device="cuda")
    binding.merge_attention(part, lse, out, lse=out_lse)
    _check(c, out, out_lse)
