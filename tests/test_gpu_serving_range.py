"""Decode attention over entries of any magnitude that the cache can hold (scale bytes 8 .. 246, any finite bf16), under
scores far from 0: what is summed in fp32 then has to be taken relative to the highest score, not to a score of 0.
Values below 2^-92 may count as 0."""
import numpy as np
import pytest

from serving_ref import HEAD, NOPE, RECORD, attention, cdiv, entries, make_cache, make_tables

pytestmark = pytest.mark.gpu

# weights between 2^-29 and 2^29, for which a reference of 0 would do, and some that pass 2^32
# (A product of a weight, down to 2^-32 of the sum it is divided by, with a value is 0 at the latest below 2^-126.)
LOST = 2.0 ** -93
SCORES = {20: [-20.0, -14.0, -1.0, 0.0, 1.0, 14.0, 20.0], 70: [-70.0, -20.0, -1.0, 0.0, 1.0, 20.0, 70.0]}


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


def _bf16(x):
    """bf16 bits of values that are exact in it."""
    bits = np.asarray(x, np.float32).view(np.uint32)
    assert not (bits & 0xffff).any()
    return (bits >> 16).astype(np.uint16)


def _record(cache, block, table, r, j):
    """Views of entry j of request r: codes, rope values (bf16 bits), scale bytes."""
    flat, off = cache[table[r, j // block]].reshape(-1), j % block
    rec = flat[off * RECORD:(off + 1) * RECORD]
    return rec[:NOPE], rec[NOPE:].view(np.uint16), flat[block * RECORD + off * 8:][:7]


def _run(binding, q, cache, block, table, lens, out, sink=None):
    import torch
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    binding.decode_attention(q, _cuda(cache), block, _cuda(table), _cuda(np.array(lens, np.int32)), 1.0, out, lse=lse, sink=sink)
    assert binding.device_errors(clear=True) == 0
    return lse


@pytest.mark.parametrize("reach", [20, 70])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("heads", [7, 28, 70])
def test_one_entry_of_any_magnitude_is_the_result(binding, heads, f32, reach):
    """Every head's score is that of its query's only column, rope column 0, where every entry holds 1."""
    import torch
    rng = np.random.default_rng([61, heads])
    scales = list(range(8, 247, 7)) + [72, 71, 143, 144, 175, 176, 181, 246]
    tops = [2.0 ** 127 * (2 - 2.0 ** -7), 2.0 ** 25, 2.0 ** 24, 2.0 ** 63, 2.0 ** 64, 2.0 ** 100, 2.0 ** -64, 2.0 ** -65, 2.0 ** -100,
            2.0 ** -126, 0.0]
    R, block = len(scales) + 2 * len(tops), 4
    cache, table = make_cache(rng, R, block), np.arange(R, dtype=np.int32)[:, None]
    codes = np.array([b for b in range(256) if b & 127 != 127], np.uint8)
    for r in range(R):
        nope, rope, scale = _record(cache, block, table, r, 0)
        nope[:] = np.resize(np.roll(codes, 31 * r), NOPE)
        if r < len(scales):
            # one group alone, or all
            scale[:] = scales[r] if r % 3 else 118
            scale[r % 7] = scales[r]
        else:
            rope[:] = _bf16(rng.integers(-128, 128, 64) / 64.0)
            top = tops[(r - len(scales)) // 2]
            at = 1 + (9 * r) % 63 if r % 2 else slice(1, 64)
            rope[at] = _bf16(top if r % 4 < 2 else -top)
        rope[0] = _bf16(1.0)
    q = torch.zeros(R, heads, HEAD, dtype=torch.bfloat16, device="cuda")
    q[:, :, NOPE] = torch.tensor(np.resize(SCORES[reach], heads), device="cuda").to(torch.bfloat16)
    out = torch.full((R, heads, HEAD), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    lse = _run(binding, q, cache, block, table, [1] * R, out)
    got, scores = out.double().cpu().numpy(), np.resize(SCORES[reach], heads)
    for r in range(R):
        want = entries(cache, block, table[r], 1)[0]
        real = np.abs(want) < 2.0 ** 128 * (1 - 2.0 ** -9)  # (codes of 256 and more overflow bf16 with a byte of 246)
        for h in range(heads):
            if f32:
                # weight times value is exact (8 bits each); the weight's reciprocal and its product with that are
                # rounded, 2^-24 each, where the weight is not 1
                assert (np.abs(got[r, h, real] - want[real]) <= LOST + (2.0 ** -23 + 2.0 ** -48) * np.abs(want[real])).all(), (r, h)
            else:
                exact = real & ((np.abs(want) >= 2.0 ** -92) | (np.abs(scores[h]) == 0))
                assert np.array_equal(got[r, h, exact], want[exact]), (r, h)
                assert (np.abs(got[r, h, real] - want[real]) <= LOST + 2.0 ** -8 * np.abs(want[real])).all(), (r, h)
    # log2 and back: a few roundings of the score
    score = q[:, :, NOPE].double().cpu().numpy()
    assert (np.abs(lse.double().cpu().numpy() - score) <= 2.0 ** -22 * np.abs(score)).all()


@pytest.mark.parametrize("reach", [20, 70])
@pytest.mark.parametrize("where", [0, 5, 63, 64, 130, 260, 899])
@pytest.mark.parametrize("big", [2.0 ** 100, -2.0 ** 126, 2.0 ** -100])
def test_one_far_entry_among_others(binding, where, big, reach):
    """An entry of another magnitude in the first tile of a request or behind it, of a request that one CTA takes or
    several share, with a score above, among or below the others'."""
    import torch
    rng = np.random.default_rng([62, where])
    heads, block, lens = 20, 64, [900, 70, 260, 131]
    pages = sum(cdiv(n, block) for n in lens)
    cache, table = make_cache(rng, pages, block), make_tables(rng, lens, block, pages)
    for r, n in enumerate(lens):
        for j in range(n):
            nope, rope, scale = _record(cache, block, table, r, j)
            rope[0] = _bf16(rng.integers(-16, 17) / 16.0)
        nope, rope, scale = _record(cache, block, table, r, min(where, n - 1))
        rope[0] = _bf16(-1.0 + r % 3)          # scores of -q, 0 or q
        rope[5:9] = _bf16(big)
        rope[11] = _bf16(-big)
        scale[2] = 127 + int(np.log2(abs(big))) - (9 if abs(big) > 1 else 0)
    q = torch.zeros(4, heads, HEAD, dtype=torch.bfloat16, device="cuda")
    q[:, :, NOPE] = torch.tensor(np.resize(SCORES[reach], heads), device="cuda").to(torch.bfloat16)
    out = torch.full((4, heads, HEAD), 7.0, device="cuda")
    lse = _run(binding, q, cache, block, table, lens, out)
    q64, out, lse = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    for r, n in enumerate(lens):
        k = entries(cache, block, table[r], n)
        want, want_lse, tol, tol_lse = attention(q64[r], k, 1.0, out_half=2.0 ** -24)
        # out = sum_j w_j (1 + e_j) k_j / sum_j w_j (1 + e_j), |e_j| <= 2^-8: off by up to 2^-8 sum_j p_j |k_j| for the e_j
        # above (in tol) and 2^-8 |out| for those below, which one entry that outweighs a column's others can feel in
        # full; 1 / (1 + e) leaves 2^-6 of that. A weight below 2^-126 of the highest is 0 in fp32.
        rounded = 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(want)
        off = np.abs(out[r] - want) - (tol + rounded + LOST + 2.0 ** -126 * np.abs(k).sum(0))
        assert np.isfinite(out[r]).all() and (off <= 0).all(), (r, np.unravel_index(off.argmax(), off.shape), off.max())
        assert (np.abs(lse[r] - want_lse) <= tol_lse).all(), r
