"""How the operators around the compressor are called: under capture, on several streams at once, with pages that
requests share, out of views and into them."""
import numpy as np
import pytest

from serving_ref import HEAD, attention, cdiv, entries, extend, make_cache, make_tables, slot_maps

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


def _decode_args(rng, lens, heads, block=64):
    import torch
    pages = sum(cdiv(int(n), block) for n in lens) + 1
    cache, table = make_cache(rng, pages, block), make_tables(rng, lens, block, pages)
    q = torch.from_numpy(rng.standard_normal((len(lens), heads, HEAD)).astype(np.float32)).to(torch.bfloat16).cuda()
    return cache, table, (q, _cuda(cache), block, _cuda(table), _cuda(np.array(lens, np.int32)), HEAD ** -0.5)


def _check_decode(cache, table, args, out, lse):
    q, block, lens, scale = args[0].double().cpu().numpy(), args[2], args[4].tolist(), args[5]
    for r, n in enumerate(lens):
        want, want_lse, tol, tol_lse = attention(q[r], entries(cache, block, table[r], n), scale, None)
        assert (np.abs(out[r].double().cpu().numpy() - want) <= tol).all(), r
        got = lse[r].double().cpu().numpy()
        assert ((got == want_lse) | (np.abs(got - want_lse) <= tol_lse)).all(), r


def _maps(T, R):
    import torch
    i32, i64 = torch.int32, torch.int64
    z = lambda n, t: torch.full((n,), -5, dtype=t, device="cuda")
    return {"query_start": z(R + 1, i32), "token_to_req_indices": z(T, i32), "positions": z(T, i64), "slot_mapping": z(T, i64),
            "kv_slot_mapping": z(T, i64), "kv_lens": z(R, i32)}


def test_first_call_on_a_captured_stream_is_refused(binding):
    """A stream without its error word: C128_ERR_CAPTURE and nothing enqueued; after reserve_workspace it is captured."""
    import torch
    rng = np.random.default_rng(41)
    cache, table, args = _decode_args(rng, [70, 3], 16)
    out, lse = torch.zeros_like(args[0]), torch.zeros(2, 16, device="cuda")
    lens, new, maps = _cuda(np.array([9, 5], np.int32)), _cuda(np.array([1, 2], np.int32)), _maps(5, 2)
    held, taken = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    blocks, free = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda")
    ws = torch.empty(binding.decode_attention_workspace(16), dtype=torch.uint8, device="cuda")
    calls = [lambda: binding.extend_block_tables(lens, held, blocks, free, taken, 1, 8),
             lambda: binding.build_slot_maps(lens, new, blocks, 8, blocks, 8, 128, **maps),
             lambda: binding.decode_attention(*args, out, lse=lse, workspace=ws)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        marker = held + 1  # a graph of its own: an empty one may not be replayed
        for call in calls:
            with pytest.raises(binding.C128Error) as e:
                call()
            assert e.value.status == 11
    g.replay()
    torch.cuda.synchronize()
    assert int(taken) == 0 and bool((out == 0).all()) and bool((maps["positions"] == -5).all()) and int(marker.sum()) == 2
    binding.reserve_workspace(1, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for call in calls:
            call()
    assert int(taken) == 0  # captured, not run
    g.replay()
    torch.cuda.synchronize()
    assert binding.device_errors(s, clear=True) == 0
    assert int(taken) == 3 and held.tolist() == [2, 1] and blocks.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]]
    want, bits = slot_maps(np.array([9, 5], np.int32), np.array([1, 2], np.int32), blocks.cpu().numpy(), 8,
                           blocks.cpu().numpy(), 8, 128, 5)
    assert bits == 0 and all(np.array_equal(maps[k].cpu().numpy(), v) for k, v in want.items())
    _check_decode(cache, table, args, out, lse)
    g.replay()  # nothing has grown: the same again
    torch.cuda.synchronize()
    assert int(taken) == 3 and held.tolist() == [2, 1]
    binding.release_stream(s)


def test_two_streams_at_once(binding):
    """Different decode calls (and the tables' calls between them) on two streams, unsynchronised: each as alone."""
    import torch
    rng = np.random.default_rng(42)
    work = []
    for lens, heads in (([900, 1, 64, 3000], 64), ([5000, 70], 20)):
        cache, table, args = _decode_args(rng, lens, heads)
        out, lse = torch.zeros_like(args[0]), torch.zeros(len(lens), heads, device="cuda")
        binding.decode_attention(*args, out, lse=lse)
        assert binding.device_errors(clear=True) == 0
        _check_decode(cache, table, args, out, lse)
        work.append((torch.cuda.Stream(), args, out, lse, len(lens), heads))
    torch.cuda.synchronize()
    outs = [[], []]
    for rep in range(30):
        for k, (s, args, out, lse, R, heads) in enumerate(work):
            with torch.cuda.stream(s):
                held, taken = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
                blocks = torch.zeros(R, 100, dtype=torch.int32, device="cuda")
                free = torch.arange(R * 100, dtype=torch.int32, device="cuda")
                binding.extend_block_tables(args[4], held, blocks, free, taken, 1, 64)
                o, l = torch.zeros_like(out), torch.zeros_like(lse)
                binding.decode_attention(*args, o, lse=l)
                outs[k].append((o, l, held, taken))
    torch.cuda.synchronize()
    for k, (s, args, out, lse, R, heads) in enumerate(work):
        assert binding.device_errors(s, clear=True) == 0
        need = [cdiv(n, 64) for n in args[4].tolist()]
        for o, l, held, taken in outs[k]:
            assert torch.equal(o, out) and torch.equal(l, lse)
            assert held.tolist() == need and int(taken) == sum(need)


def test_shared_and_repeated_pages(binding):
    """Requests that share pages (a common prefix), and one whose table lists a page twice."""
    import torch
    rng = np.random.default_rng(43)
    block, heads, lens = 64, 24, [200, 190, 256, 64]
    cache = make_cache(rng, 6, block)
    table = np.array([[4, 2, 0, 5], [4, 2, 0, 1], [3, 3, 1, 3], [4, -1, -1, -1]], np.int32)
    q = torch.from_numpy(rng.standard_normal((4, heads, HEAD)).astype(np.float32)).to(torch.bfloat16).cuda()
    args = (q, _cuda(cache), block, _cuda(table), _cuda(np.array(lens, np.int32)), HEAD ** -0.5)
    out, lse = torch.zeros_like(q), torch.zeros(4, heads, device="cuda")
    binding.decode_attention(*args, out, lse=lse)
    assert binding.device_errors(clear=True) == 0
    _check_decode(cache, table, args, out, lse)


def test_tables_into_views_and_free_lists_behind_an_offset(binding):
    """Lengths at an odd place (no 16-byte loads), table rows inside a wider buffer, taken in the middle of the list."""
    import torch
    rng = np.random.default_rng(44)
    R, MB = 77, 9
    lens = rng.integers(0, MB * 8 + 1, R).astype(np.int32)
    held = np.minimum(rng.integers(0, 4, R), [cdiv(int(n), 8) for n in lens]).astype(np.int32)
    table = rng.integers(0, 1 << 20, (R, MB)).astype(np.int32)
    free = rng.permutation(1000).astype(np.int32)
    want = extend(lens, held, table, free, 123, 1, 8)
    odd = lambda a: torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), _cuda(a)])[1:]
    wide = torch.full((R, MB + 3), -7, dtype=torch.int32, device="cuda")
    t = wide[:, 2:2 + MB]
    t.copy_(_cuda(table))
    h, k = odd(held), torch.tensor([123], dtype=torch.int64, device="cuda")
    binding.extend_block_tables(odd(lens), h, t, odd(free), k, 1, 8)
    assert binding.device_errors(clear=True) == want[3]
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(h.cpu().numpy(), want[1]) and int(k) == want[2]
    assert bool((wide[:, :2] == -7).all()) and bool((wide[:, 2 + MB:] == -7).all())


def test_decode_over_an_empty_cache(binding):
    """No block at all: zeros and -inf (the sink), and a request that claims entries has them left out."""
    import torch
    q = torch.ones(3, 20, HEAD, dtype=torch.bfloat16, device="cuda")
    cache = torch.empty(0, 64, 584, dtype=torch.uint8, device="cuda")
    table = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    sink = torch.linspace(-3, 3, 20, device="cuda")
    for lens, bits in (([0, 0, 0], 0), ([0, 200, 64], 4)):
        for with_sink in (None, sink):
            out, lse = torch.full_like(q, 7), torch.full((3, 20), 7.0, device="cuda")
            binding.decode_attention(q, cache, 64, table, _cuda(np.array(lens, np.int32)), 0.05, out, lse=lse, sink=with_sink)
            assert binding.device_errors(clear=True) == bits
            assert bool((out == 0).all())
            if with_sink is None:
                assert bool((lse == -np.inf).all())
            else:
                # log2 and back of the sink: a few roundings of a value of 3
                assert bool(((lse - sink).abs() <= 2.0 ** -20).all())


@pytest.mark.parametrize("lens,heads", [([64], 16), ([300, 64, 5, 700], 40)])
def test_calls_follow_one_another_without_gaps(binding, lens, heads):
    """Tables rewritten between attention calls that are launched back to back (each launch starts before the one before
    it has ended): every call sees the table that was written right before it, one of two sets of pages."""
    import torch
    rng = np.random.default_rng([45, heads])
    block, R = 64, len(lens)
    need = [cdiv(n, block) for n in lens]
    cache = make_cache(rng, 2 * sum(need), block)
    pages = rng.permutation(2 * sum(need)).astype(np.int32).reshape(2, -1)
    q = torch.from_numpy(rng.standard_normal((R, heads, HEAD)).astype(np.float32)).to(torch.bfloat16).cuda()
    lens_gpu, held, taken = _cuda(np.array(lens, np.int32)), _cuda(np.zeros(R, np.int32)), torch.zeros(1, dtype=torch.int64, device="cuda")
    table = torch.full((R, max(need)), -1, dtype=torch.int32, device="cuda")
    held_out, taken_out = torch.empty_like(held), torch.empty_like(taken)
    fill = [binding.PreparedOp("extend_block_tables", lens_gpu, held, table, _cuda(pages[k]), taken, 1, block, held_out=held_out,
                               taken_out=taken_out) for k in range(2)]
    cache_gpu = _cuda(cache)
    outs = [(torch.zeros_like(q), torch.zeros(R, heads, device="cuda")) for _ in range(40)]
    calls = [binding.PreparedOp("decode_attention", q, cache_gpu, block, table, lens_gpu, HEAD ** -0.5, o, lse=l) for o, l in outs]
    torch.cuda.synchronize()
    for k, call in enumerate(calls):
        fill[k % 2]()
        call()
    torch.cuda.synchronize()
    assert binding.device_errors(clear=True) == 0
    for k in range(2):
        rows = np.full((R, max(need)), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            rows[r, :n] = pages[k][at:at + n]
            at += n
        _check_decode(cache, rows, (q, None, block, None, lens_gpu, HEAD ** -0.5), *outs[k])
        for o, l in outs[k::2]:
            assert torch.equal(o, outs[k][0]) and torch.equal(l, outs[k][1])
