"""Decode attention without a workspace on a stream that is not torch's current one: its scratch is neither memory that
queued work on the current stream still uses, nor handed out again while the call runs."""
import numpy as np
import pytest

from serving_ref import HEAD, attention, cdiv, entries, make_cache, make_tables

pytestmark = pytest.mark.gpu

SLEEP = 200000000  # cycles: about 0.1 s


@pytest.fixture(scope="module")
def binding():
    from deepseek_v4_sparse_c128_gb300 import binding as b
    from deepseek_v4_sparse_c128_gb300 import build
    build.build()
    b.load()
    b.device_errors(clear=True)
    return b


def _case():
    import torch
    rng = np.random.default_rng(71)
    lens, heads, block = [5000, 77], 64, 64
    pages = sum(cdiv(n, block) for n in lens)
    cache, table = make_cache(rng, pages, block), make_tables(rng, lens, block, pages)
    q = torch.from_numpy((2 * rng.standard_normal((2, heads, HEAD))).astype(np.float32)).to(torch.bfloat16).cuda()
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = (q, cuda(cache), block, cuda(table), cuda(np.array(lens, np.int32)), HEAD ** -0.5)
    want = [attention(q[r].double().cpu().numpy(), entries(cache, block, table[r], n), HEAD ** -0.5) for r, n in enumerate(lens)]

    def check(out, lse):
        for r in range(2):
            assert (np.abs(out[r].double().cpu().numpy() - want[r][0]) <= want[r][2]).all()
            assert (np.abs(lse[r].double().cpu().numpy() - want[r][1]) <= want[r][3]).all()
    return args, torch.full_like(q, 7), torch.full((2, heads), 7.0, device="cuda"), check


def _call(binding, how, args, out, lse, stream):
    """A call of each kind; what it returns has to live as long as the caller wants."""
    if how == "prepared":
        op = binding.PreparedOp("decode_attention", *args, out, lse=lse, stream=stream)
        op()
        return op
    return binding.decode_attention(*args, out, lse=lse, stream=stream if how == "stream" else stream.cuda_stream)


@pytest.mark.parametrize("how", ["stream", "handle", "prepared"])
def test_scratch_is_not_memory_that_the_current_stream_still_reads(binding, how):
    import torch
    args, out, lse, check = _case()
    n = binding.decode_attention_workspace(64)
    s = torch.cuda.Stream()
    _call(binding, how, args, out, lse, s)  # the stream's error word
    torch.cuda.synchronize()
    out.fill_(7)
    mine = torch.full((n,), 5, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    copy = mine.clone()  # behind the sleep
    del mine
    op = _call(binding, how, args, out, lse, s)
    torch.cuda.synchronize()
    assert bool((copy == 5).all())
    assert binding.device_errors(s, clear=True) == 0
    check(out, lse)
    del op


@pytest.mark.parametrize("how", ["stream", "handle", "prepared"])
def test_scratch_of_a_call_in_flight_is_not_handed_out(binding, how):
    import torch
    args, out, lse, check = _case()
    n = binding.decode_attention_workspace(64)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    op = _call(binding, how, args, out, lse, s)
    del op  # the call has not begun
    others = [torch.full((n,), 9, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((t == 9).all()) for t in others)
    assert binding.device_errors(s, clear=True) == 0
    check(out, lse)


def test_a_handle_of_0_is_the_default_stream(binding):
    """The call runs on the default stream while another is current: its scratch is the default stream's."""
    import torch
    args, out, lse, check = _case()
    n = binding.decode_attention_workspace(64)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        binding.decode_attention(*args, out, lse=lse, stream=0)
        torch.cuda.synchronize()
        out.fill_(7)
        mine = torch.full((n,), 5, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(SLEEP)
        copy = mine.clone()
        del mine
        op = binding.PreparedOp("decode_attention", *args, out, lse=lse, stream=0)
        op()
        del op
        others = [torch.full((n,), 9, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert bool((copy == 5).all()) and all(bool((t == 9).all()) for t in others)
    assert binding.device_errors(0, clear=True) == 0
    check(out, lse)
