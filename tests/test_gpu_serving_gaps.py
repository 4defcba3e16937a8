"""Block tables, per-token arrays and the compressor's call launched back to back, two steps in turn over the same
arrays: each kernel may start while the ones before it still run, and every call has to see the arrays that were written
right before it. Each of the compressor's kernels is behind one of the cases."""
import numpy as np
import pytest

from deepseek_v4_sparse_c128_gb300 import inputs
from serving_ref import cdiv, make_cache, make_tables

pytestmark = pytest.mark.gpu

SLOT_BYTES = {0: 584, 1: 132, 2: 68}


@pytest.fixture(scope="module")
def binding():
    from deepseek_v4_sparse_c128_gb300 import binding as b
    from deepseek_v4_sparse_c128_gb300 import build
    build.build()
    b.load()
    b.device_errors(clear=True)
    return b


@pytest.mark.parametrize("head,ratio,overlap,fmt,state_block,requests,most_new", [
    (512, 128, 0, 0, 8, 3, 40), (512, 128, 0, 0, 8, 5, 200), (512, 128, 0, 0, 16, 5, 200), (512, 128, 0, 0, 8, 30, 300),
    (512, 4, 1, 0, 8, 4, 30), (512, 4, 1, 0, 8, 30, 300), (128, 4, 1, 1, 8, 4, 30), (128, 4, 1, 2, 8, 30, 300),
    (128, 128, 0, 2, 8, 4, 60), (128, 128, 0, 1, 8, 30, 300), (128, 128, 0, 2, 4, 30, 300), (512, 128, 0, 0, 4, 20, 300),
])
def test_steps_follow_one_another_without_gaps(binding, head, ratio, overlap, fmt, state_block, requests, most_new):
    import torch
    rng = np.random.default_rng([81, head, ratio, fmt, state_block, requests])
    longest, kv_block = 1000, 4
    new = rng.integers(0, most_new + 1, (2, requests)).astype(np.int32)
    lens = np.minimum(new + rng.integers(0, longest, (2, requests)), longest).astype(np.int32)
    lens[:, 0], new[:, 0] = 5 * 128, min(most_new, 128)     # a window of 128 ends in both steps
    tokens = int(new.sum(1).max()) + 3
    columns, kv_columns = cdiv(longest, state_block), cdiv(longest // ratio, kv_block) + 1
    state_blocks = max(sum(cdiv(int(n), state_block) for n in row) for row in lens)
    kv_blocks = max(sum(cdiv(int(n) // ratio, kv_block) for n in row) for row in lens)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64, device="cuda")
    width = head * (1 + overlap)
    state = inputs.draw_state_rows(91, state_blocks, state_block, width, "cuda")
    rms_w = cuda((1 + 0.1 * rng.standard_normal(head)).astype(np.float32))
    cos_sin = cuda(inputs._cos_sin_cache(longest))
    table, kv_table = i32(requests, columns), i32(requests, kv_columns)
    maps = {"query_start": i32(requests + 1), "token_to_req_indices": i32(tokens), "positions": i64(tokens),
            "slot_mapping": i64(tokens), "kv_slot_mapping": i64(tokens), "kv_lens": i32(requests)}
    cfg = binding.config(head, ratio, overlap, width, fmt)
    zero, held_out, nothing, taken_out = i32(requests), i32(requests), i64(1), i64(1)
    P = binding.PreparedOp
    steps = []
    for k in range(2):
        n = cuda(lens[k])
        steps.append([
            P("extend_block_tables", n, zero, table, cuda(rng.permutation(state_blocks).astype(np.int32)), nothing, 1, state_block,
              held_out=held_out, taken_out=taken_out),
            P("extend_block_tables", n, zero, kv_table, cuda(rng.permutation(kv_blocks).astype(np.int32)), nothing, ratio, kv_block,
              held_out=held_out, taken_out=taken_out),
            P("build_slot_maps", n, cuda(new[k]), table, state_block, kv_table, kv_block, ratio, **maps)])

    def compress(cache):
        return binding.PreparedCall(maps["token_to_req_indices"], maps["positions"], maps["slot_mapping"], table, state, rms_w,
                                    1e-6, cos_sin, cache, maps["kv_slot_mapping"], kv_block, cfg=cfg)

    caches = torch.zeros(18, kv_blocks, kv_block, SLOT_BYTES[fmt], dtype=torch.uint8, device="cuda")
    calls = [compress(c) for c in caches]
    for k in range(2):                                       # each step by itself
        for call in (*steps[k], calls[k]):
            call()
            torch.cuda.synchronize()
    assert not torch.equal(caches[0], caches[1])
    for rep in range(2, 18):
        for call in (*steps[rep % 2], calls[rep]):
            call()
    torch.cuda.synchronize()
    assert binding.device_errors(clear=True) == 0
    for rep in range(2, 18):
        assert torch.equal(caches[rep], caches[rep % 2]), rep


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("requests,heads", [(1, 16), (5, 40), (60, 8)])
def test_attention_and_merge_follow_one_another_without_gaps(binding, requests, heads, f32):
    """Two queries in turn through attention over two caches and the merge, the partial results in the same tensors:
    every merge joins what was written right before it, out of place and in place."""
    import torch
    rng = np.random.default_rng([82, requests, heads])
    block, lens = 64, rng.integers(1, 700, (2, requests)).astype(np.int32)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    caches, tables = [], []
    for k in range(2):
        pages = sum(cdiv(int(n), block) for n in lens[k])
        caches.append(cuda(make_cache(rng, pages, block)))
        tables.append(cuda(make_tables(rng, lens[k], block, pages)))
    q = [torch.from_numpy((2 * rng.standard_normal((requests, heads, 512))).astype(np.float32)).to(torch.bfloat16).cuda()
         for _ in range(2)]
    kind = torch.float32 if f32 else torch.bfloat16
    part = torch.zeros(2, requests, heads, 512, dtype=kind, device="cuda")
    part_lse = torch.zeros(2, requests, heads, device="cuda")
    lens_gpu = [cuda(n) for n in lens]
    P = binding.PreparedOp
    attend = [[P("decode_attention", q[i], caches[k], block, tables[k], lens_gpu[k], 512 ** -0.5, part[k], lse=part_lse[k])
               for k in range(2)] for i in range(2)]
    reps = 24
    outs = torch.zeros(reps, requests, heads, 512, dtype=kind, device="cuda")
    lses = torch.zeros(reps, requests, heads, device="cuda")
    merges = [P("merge_attention", part, part_lse, outs[r], lse=lses[r]) for r in range(reps)]
    in_place = P("merge_attention", part, part_lse, part[1], lse=part_lse[1])
    for r in range(2):                                       # each by itself
        for call in (*attend[r], merges[r]):
            call()
            torch.cuda.synchronize()
    assert not torch.equal(outs[0], outs[1])
    for r in range(2, reps):
        for call in (*attend[r % 2], merges[r]):
            call()
        in_place()
        outs[r][0, 0].copy_(part[1][0, 0])                   # a row of the merge in place
    torch.cuda.synchronize()
    assert binding.device_errors(clear=True) == 0
    for r in range(2, reps):
        assert torch.equal(outs[r], outs[r % 2]) and torch.equal(lses[r], lses[r % 2]), r
