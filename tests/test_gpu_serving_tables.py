"""c128_extend_block_tables and c128_build_slot_maps against plain loops (whole numbers, so equal), at the sizes
where a prefix sum over rounds of 512 or 1024 requests and tiles of blocks or tokens can go wrong."""
import numpy as np
import pytest

from serving_ref import cdiv, extend, make_tables, slot_maps

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


def _run_extend(binding, lens, held, table, free, taken, ratio, block, in_place=False, pad=0):
    import torch
    R, MB = table.shape
    wide = torch.full((R, MB + pad), -7, dtype=torch.int32, device="cuda")
    wide[:, :MB] = _cuda(table)
    t = wide[:, :MB]
    h, k = _cuda(held), torch.tensor([taken], dtype=torch.int64, device="cuda")
    ho, ko = (None, None) if in_place else (torch.full_like(h, -9), torch.full_like(k, -9))
    binding.extend_block_tables(_cuda(lens), h, t, _cuda(free), k, ratio, block, held_out=ho, taken_out=ko)
    bits = binding.device_errors(clear=True)
    if not in_place:
        assert np.array_equal(h.cpu().numpy(), held) and int(k) == taken
    assert bool((wide[:, MB:] == -7).all())
    return t.cpu().numpy(), (h if in_place else ho).cpu().numpy(), int(k if in_place else ko), bits


def _check_extend(binding, lens, held, table, free, taken, ratio, block, **kw):
    want = extend(lens, held, table, free, taken, ratio, block)
    got = _run_extend(binding, lens, held, table, free, taken, ratio, block, **kw)
    assert np.array_equal(got[0], want[0])
    assert np.array_equal(got[1], want[1])
    assert got[2:] == want[2:]
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests,longest,ratio,block", [
    (1, 1, 1, 8), (1, 100000, 1, 8), (3, 7, 1, 8), (256, 900, 1, 8), (513, 300, 4, 2), (2047, 50, 1, 3),
    (2048, 40, 1, 1), (2049, 64, 128, 1), (5000, 33, 1, 8), (7, 20001, 1, 1), (1023, 9, 1, 8), (1024, 20, 1, 8),
    (1025, 20, 1, 8), (9000, 300, 1, 1),
])
def test_extend_matches_loops(binding, requests, longest, ratio, block, in_place):
    rng = np.random.default_rng([requests, longest, ratio, block])
    lens = rng.integers(0, longest + 1, requests, dtype=np.int32)
    needed = np.array([cdiv(int(n) // ratio, block) for n in lens], np.int32)
    held = (needed * rng.random(requests)).astype(np.int32)
    held[rng.random(requests) < 0.2] = needed[rng.random(requests) < 0.2].max(initial=0)  # some hold more than they need
    cols = max(int(needed.max()), int(held.max()), 1)
    table = rng.integers(0, 1 << 30, (requests, cols), dtype=np.int32)
    taken = 5
    free = rng.permutation(int(np.maximum(needed - held, 0).sum()) + taken + 3).astype(np.int32)
    want = _check_extend(binding, lens, held, table, free, taken, ratio, block, in_place=in_place, pad=in_place * 3)
    assert want[3] == 0


def test_extend_grows_step_by_step(binding):
    """In place over many steps, as a decode loop does it: every table entry is a block given once."""
    import torch
    R, block = 37, 8
    lens = torch.randint(0, 30, (R,), dtype=torch.int32, device="cuda")
    held = torch.zeros(R, dtype=torch.int32, device="cuda")
    taken = torch.zeros(1, dtype=torch.int64, device="cuda")
    table = torch.full((R, 40), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(1000, device="cuda").to(torch.int32)
    op = binding.PreparedOp("extend_block_tables", lens, held, table, free, taken, 1, block)
    for _ in range(60):
        op()
        lens += torch.randint(0, 5, (R,), dtype=torch.int32, device="cuda")
    op()
    assert binding.device_errors(clear=True) == 0
    assert bool((held == (lens + block - 1) // block).all()) and int(taken) == int(held.sum())
    given = table[torch.arange(40, device="cuda")[None, :] < held[:, None]]
    assert sorted(given.tolist()) == sorted(free[:int(taken)].tolist())
    assert bool((table[torch.arange(40, device="cuda")[None, :] >= held[:, None]] == -1).all())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("short", [0, 1, 17, 4000])
def test_extend_out_of_blocks(binding, short, in_place):
    rng = np.random.default_rng(short)
    lens = rng.integers(0, 40, 2500, dtype=np.int32)
    held = np.zeros(2500, np.int32)
    total = sum(cdiv(int(n), 2) for n in lens)
    free = rng.permutation(total - short).astype(np.int32)
    table = np.full((2500, 20), -1, np.int32)
    want = _check_extend(binding, lens, held, table, free, 0, 1, 2, in_place=in_place)
    assert want[3] == (64 if short else 0)


def test_extend_bad_values(binding):
    lens = np.array([100, -5, 30, 2000, 16, 8, 2147483647], np.int32)
    held = np.array([0, 0, -1, 1, 2, 0, 0], np.int32)
    table = np.full((7, 16), -1, np.int32)
    free = np.arange(50, dtype=np.int32)
    want = _check_extend(binding, lens, held, table, free, 3, 1, 8)
    assert want[3] == 128 | 2
    for taken in (-1, 51):
        want = _check_extend(binding, lens, held, table, free, taken, 1, 8)
        assert want[3] == 128 | 64 | 2 and np.array_equal(want[0], table)
    # nothing to do at all
    empty = np.zeros(0, np.int32)
    assert _run_extend(binding, empty, empty, np.zeros((0, 4), np.int32), free, 7, 1, 8)[2] == 7
    _check_extend(binding, np.array([9], np.int32), np.array([0], np.int32), np.full((1, 2), -1, np.int32), empty, 0, 1, 8)


def _run_maps(binding, lens, new, st, sb, kt, kb, ratio, tokens, offset=0):
    """The outputs as numpy; `offset` shifts every output's start off its 16-byte alignment."""
    import torch
    R = len(lens)
    sizes = {"query_start": (R + 1, torch.int32), "token_to_req_indices": (tokens, torch.int32),
             "positions": (tokens, torch.int64), "slot_mapping": (tokens, torch.int64),
             "kv_slot_mapping": (tokens, torch.int64), "kv_lens": (R, torch.int32)}
    whole = {k: torch.full((n + offset + 2,), -77, dtype=t, device="cuda") for k, (n, t) in sizes.items()}
    outs = {k: whole[k][offset:offset + n] for k, (n, _) in sizes.items()}
    pads = [_cuda(np.concatenate([np.zeros(offset, np.int32), v]))[offset:] for v in (lens, new)]
    binding.build_slot_maps(*pads, _cuda(st), sb, _cuda(kt), kb, ratio, **outs)
    bits = binding.device_errors(clear=True)
    for k, (n, _) in sizes.items():
        assert bool((whole[k][:offset] == -77).all()) and bool((whole[k][offset + n:] == -77).all()), k
    return {k: v.cpu().numpy() for k, v in outs.items()}, bits


def _check_maps(binding, lens, new, st, sb, kt, kb, ratio, tokens, **kw):
    want, want_bits = slot_maps(lens, new, st, sb, kt, kb, ratio, tokens)
    got, bits = _run_maps(binding, lens, new, st, sb, kt, kb, ratio, tokens, **kw)
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    assert bits == want_bits
    return want, bits


@pytest.mark.parametrize("requests,longest,most_new,pad,ratio,sb,kb,offset", [
    (1, 1, 1, 0, 128, 8, 64, 0), (1, 1, 1, 5, 1, 8, 1, 1), (1, 5000, 5000, 0, 4, 8, 2, 0), (3, 700, 1, 2, 128, 8, 64, 1),
    (200, 3000, 1, 56, 128, 8, 64, 0), (333, 900, 40, 7, 4, 8, 2, 0), (2048, 60, 3, 0, 4, 8, 1, 0),
    (2049, 60, 3, 1000, 8, 3, 7, 3), (5000, 20, 1, 1, 2, 8, 64, 0), (64, 4000, 900, 1025, 128, 8, 64, 0),
    (511, 60, 3, 3, 4, 8, 2, 0), (512, 60, 3, 0, 128, 8, 1, 1), (513, 60, 3, 9, 4, 8, 2, 0), (1024, 90, 2, 0, 8, 8, 2, 2),
    (1025, 90, 2, 0, 8, 8, 2, 0),
])
def test_maps_match_loops(binding, requests, longest, most_new, pad, ratio, sb, kb, offset):
    rng = np.random.default_rng([requests, longest, most_new, pad])
    lens = rng.integers(1, longest + 1, requests, dtype=np.int32)
    new = np.minimum(lens, rng.integers(0, most_new + 1, requests)).astype(np.int32)
    if requests > 2:
        new[rng.integers(0, requests, requests // 3)] = 0   # requests without new tokens, some in a row
        lens[requests // 2] = new[requests // 2] = 0
    new[-1] = max(1, new[-1])
    st = make_tables(rng, lens, sb, sum(cdiv(int(n), sb) for n in lens))
    kt = make_tables(rng, lens // ratio, kb, sum(cdiv(int(n) // ratio, kb) for n in lens) + 1)
    _, bits = _check_maps(binding, lens, new, st, sb, kt, kb, ratio, int(new.sum()) + pad, offset=offset)
    assert bits == 0


def test_maps_far_positions(binding):
    """Positions up to the largest int32 and slots that pass 32 bits."""
    lens, new = np.array([2147483647, 2147483520], np.int32), np.array([130, 3], np.int32)
    big = 1 << 20
    st = np.array([[7] * 2047 + [2000000000]] * 2, np.int32)
    kt = np.array([[1, 2147483647], [5, 2147483646]], np.int32)
    want, bits = _check_maps(binding, lens, new, st, big, kt, 1 << 23, 128, 140)
    assert bits == 0 and want["slot_mapping"].max() > 1 << 50 and want["kv_slot_mapping"].max() > 1 << 50


def test_maps_bad_values(binding):
    rng = np.random.default_rng(3)
    lens = np.array([40, -3, 10, 300, 64, 16], np.int32)
    new = np.array([5, 2, 12, 200, -1, 16], np.int32)
    st = rng.integers(0, 99, (6, 20), dtype=np.int32)       # request 3 passes its end
    kt = rng.integers(0, 99, (6, 3), dtype=np.int32)
    st[5, 1] = -1
    kt[0, 0] = -4
    tokens = int(np.maximum(new, 0).sum())
    _, bits = _check_maps(binding, lens, new, st, 8, kt, 4, 4, tokens + 3)
    assert bits == 128 | 2 | 4
    # more tokens than rows: those behind are dropped
    ok = np.full((6, 60), 9, np.int32)
    _, bits = _check_maps(binding, np.abs(lens) + 20, np.abs(new), ok, 8, ok, 4, 4, 100)
    assert bits == 128
    # no request, and no row
    none = np.zeros(0, np.int32)
    _check_maps(binding, none, none, np.zeros((0, 4), np.int32), 8, np.zeros((0, 4), np.int32), 4, 4, 9)
    _check_maps(binding, lens[:1], new[:1] * 0, st[:1], 8, kt[:1], 4, 4, 0)
