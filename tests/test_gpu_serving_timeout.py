"""Decode attention after a wait that ran out, on a request that several CTAs share: what the CTA that gave up had a part
in is left as it was, and not joined from whatever the workspace held."""
import numpy as np
import pytest

from serving_ref import HEAD, attention, cdiv, entries, make_cache, make_tables

pytestmark = pytest.mark.gpu

TIMEOUT = 32


@pytest.fixture(scope="module")
def binding():
    from deepseek_v4_sparse_c128_gb300 import binding as b
    from deepseek_v4_sparse_c128_gb300 import build
    build.build()
    b.load()
    b.device_errors(clear=True)
    return b


@pytest.mark.parametrize("heads,lost", [(16, 16), (10, 10), (128, 64)])
def test_a_request_shared_with_a_cta_that_gave_up_is_left_as_it_was(binding, heads, lost):
    """CTA 0 starts request 0 and shares it with many others: with one head group all its heads are lost, with two
    groups of 64 (CTA 1 holds the second) the first 64. Every other request, and the next call, are right."""
    import torch
    rng = np.random.default_rng([51, heads])
    lens, block = [30000, 64, 500, 9000], 64
    pages = sum(cdiv(n, block) for n in lens)
    cache, table = make_cache(rng, pages, block), make_tables(rng, lens, block, pages)
    q = torch.from_numpy((2 * rng.standard_normal((4, heads, HEAD))).astype(np.float32)).to(torch.bfloat16).cuda()
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = (q, cuda(cache), block, cuda(table), cuda(np.array(lens, np.int32)), HEAD ** -0.5)
    # scratch that would be seen: finite parts, and statistics that are not -inf
    ws = torch.full((binding.decode_attention_workspace(heads) // 4,), 3.0, device="cuda").view(torch.uint8)

    def check(out, lse, first_head):
        out, lse, q64 = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
        for r, n in enumerate(lens):
            h = slice(first_head if r == 0 else 0, heads)
            if h.start == heads:
                continue
            want, want_lse, tol, tol_lse = attention(q64[r, h], entries(cache, block, table[r], n), HEAD ** -0.5)
            assert (np.abs(out[r, h] - want) <= tol).all(), r
            assert (np.abs(lse[r, h] - want_lse) <= tol_lse).all(), r

    out = torch.full((4, heads, HEAD), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, heads), 7.0, device="cuda")
    torch.cuda.synchronize()
    binding.debug_stall_decode_attention(*args, out, lse=lse, workspace=ws)
    assert binding.device_errors(clear=True) == TIMEOUT
    assert bool((out[0, :lost] == 7).all()) and bool((lse[0, :lost] == 7).all())
    check(out, lse, lost)
    binding.decode_attention(*args, out, lse=lse, workspace=ws)
    assert binding.device_errors(clear=True) == 0
    check(out, lse, 0)
