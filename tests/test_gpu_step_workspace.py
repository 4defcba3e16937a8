"""Workspaces of the two attentions over a paged cache: each takes its own size, short windows none, and none takes more than it says."""
import ctypes

import numpy as np
import pytest
import torch

import serving_ref as sref
from deepseek_v4_sparse_c128_gb300 import binding
from test_gpu_step_window import Case, consecutive, drafts, with_a_prompt

pytestmark = pytest.mark.gpu
ARG = 7


def guarded(n):
    """n bytes on a 256-byte boundary with others before and behind: (the bytes, all of them)."""
    whole = torch.full((n + 512,), 123, dtype=torch.uint8, device="cuda")
    start = -whole.data_ptr() % 256 or 256
    return whole[start:start + n], whole


def untouched(ws, whole):
    at = ws.data_ptr() - whole.data_ptr() if ws.numel() else 256
    return bool((whole[:at] == 123).all()) and bool((whole[at + ws.numel():] == 123).all())


def test_sizes():
    """What decode attention keeps: a task a CTA, and of two parts a CTA column the results and statistics of its heads, in sixteens
    up to a group of 64. Windows of up to 16 heads: room for 64 rows."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    for heads in (1, 5, 16, 17, 32, 64):
        rows = 2 * sms * sref.cdiv(heads, 16) * 16
        size = up(16 * sms) + up(4 * rows) + 2048 * rows
        assert binding.decode_attention_workspace(heads) == size
        assert binding.window_attention_workspace(heads, 128, 8) == 0
        assert binding.window_attention_workspace(heads, 128, 9) == (binding.decode_attention_workspace(64) if heads <= 16 else size)
    for heads in (65, 128, 1024):
        assert binding.window_attention_workspace(heads, 136) == 0
        assert binding.window_attention_workspace(heads, 1 << 20, 1 << 20) == binding.decode_attention_workspace(heads)


@pytest.mark.parametrize("heads", [1, 16, 17, 65])
def test_decode_attention_stays_within_its_own(heads):
    rng = np.random.default_rng(heads)
    lens, block = [9000, 64, 500, 20000], 16
    pages = sum(sref.cdiv(n, block) for n in lens)
    cache, table = sref.make_cache(rng, pages, block), sref.make_tables(rng, lens, block, pages)
    q = torch.from_numpy(rng.standard_normal((4, heads, 512))).bfloat16()
    ws, whole = guarded(binding.decode_attention_workspace(heads))
    out = torch.zeros(4, heads, 512, dtype=torch.bfloat16, device="cuda")
    binding.decode_attention(q.cuda(), torch.from_numpy(cache).cuda(), block, torch.from_numpy(table).cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), 512 ** -0.5, out, workspace=ws)
    assert binding.device_errors() == 0 and untouched(ws, whole)
    for r, n in enumerate(lens):
        want, _, tol, _ = sref.attention(q[r].double().numpy(), sref.entries(cache, block, table[r], n), 512 ** -0.5)
        assert (np.abs(out[r].double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("H", [64, 5, 100])
def test_short_windows_take_none(H):
    c = Case(110, consecutive(0, 100, 40), [140], H, 100, 36, 8)
    dev = [torch.from_numpy(a).cuda() for a in (c.cache, c.table, c.req, c.pos, c.slots)]
    out, lse = torch.empty(40, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(40, H, device="cuda")
    for ws in (torch.empty(0, dtype=torch.uint8, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda"), None):
        out.fill_(3), lse.fill_(7)
        binding.window_attention(c.q.cuda(), dev[0], c.block, *dev[1:], 100, c.scale, out, first=36, lse=lse, workspace=ws)
        assert binding.device_errors() == 0
        c.check(out, lse, tokens=range(0, 40, 7))
    op = binding.PreparedOp("window_attention", c.q.cuda(), dev[0], c.block, *dev[1:], 100, c.scale, out, first=36, lse=lse)
    assert [t.numel() for t in op._keep[-1]] == [0]  # (what the call took for itself)


def test_long_windows_of_few_heads_with_either_size():
    """Tokens that follow one another go together where there is room for it, else each goes alone; a C caller may give the size of
    decode attention, and what it gave is not written past."""
    c = Case(111, **with_a_prompt(drafts([400, 600], [8, 8]), [408, 608], 180, 2, H=12, block=8, sink=True))
    dev = [torch.from_numpy(a).cuda() for a in (c.cache, c.table, c.req, c.pos, c.slots)]
    small, large = binding.decode_attention_workspace(12), binding.window_attention_workspace(12, 180, 2)
    assert small < large
    tokens = [*range(16), *range(16, len(c.tokens), 37)]
    q, sink, T = c.q.cuda(), c.sink.cuda(), len(c.tokens)
    results = []
    for n in (small, large - 1, large):
        ws, whole = guarded(n)
        out = torch.full((T, 12, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, 12), 7.0, device="cuda")
        a = binding._refs(q, dev[0], *dev[1:], sink, out, lse, ws)
        rc = binding.lib().c128_window_attention(*a[:2], c.block, *a[2:6], c.window, c.first, c.scale, *a[6:],
                                                 ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert rc == 0 and binding.device_errors() == 0 and untouched(ws, whole)
        c.check(out, lse, tokens=tokens)
        results.append(out)
    assert torch.equal(results[0], results[1])
    # the Python call takes its own where it is given the smaller, and that is left alone
    ws, whole = guarded(small)
    out, lse = torch.empty_like(results[2]), torch.empty(T, 12, device="cuda")
    binding.window_attention(q, dev[0], c.block, *dev[1:], c.window, c.scale, out, first=c.first, lse=lse, sink=sink, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, results[2]) and bool((whole == 123).all())


@pytest.mark.parametrize("H", [12, 40])
def test_less_than_either_takes_is_refused(H):
    c = Case(112, consecutive(0, 300, 9), [309], H, 200, 0, 8)
    dev = [torch.from_numpy(a).cuda() for a in (c.cache, c.table, c.req, c.pos, c.slots)]
    out = torch.full((9, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(binding.decode_attention_workspace(H) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(binding.C128Error) as e:
        binding.window_attention(c.q.cuda(), dev[0], c.block, *dev[1:], 200, c.scale, out, workspace=ws)
    assert e.value.status == ARG
    torch.cuda.synchronize()
    assert bool((out == 3).all())
