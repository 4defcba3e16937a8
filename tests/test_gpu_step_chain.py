"""The operators as a model's step uses them together: tables of slots, rotations, queries and keys, attention over the
window and over the compressed cache, their merge, and the position taken out again; eager and from a graph."""
import math

import numpy as np
import pytest
import torch

import serving_ref as sref
import step_ref as ref
from deepseek_v4_sparse_c128_gb300 import binding

pytestmark = pytest.mark.gpu
H, WINDOW, FIRST, EPS, BLOCK, RATIO, KV_BLOCK = 12, 24, 2, 1e-6, 16, 8, 4


class Step:
    """Three requests: a prompt from its beginning, a part of one, one new token; two padded rows."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        cuda = lambda a, t=torch.int32: torch.tensor(np.ascontiguousarray(a), dtype=t, device="cuda")  # noqa: E731
        self.lens, self.new = [40, 70, 33], [40, 9, 1]
        T = sum(self.new) + 2
        self.T = T
        self.seq_lens, self.query_lens = cuda(self.lens), cuda(self.new)
        self.table_np = sref.make_tables(rng, self.lens, BLOCK, 12)
        self.state_table, self.table = cuda(self.table_np), cuda(self.table_np)
        kv = [n // RATIO for n in self.lens]
        self.kv_table_np = sref.make_tables(rng, [n // RATIO + 1 for n in self.lens], KV_BLOCK, 9)
        self.kv_table = cuda(self.kv_table_np)
        self.kv_cache_np = sref.make_cache(rng, 9, KV_BLOCK)
        self.kv_cache = torch.from_numpy(self.kv_cache_np).cuda()
        # the window's cache holds what earlier steps stored
        self.cache_np = sref.make_cache(rng, 12, BLOCK)
        self.cache = torch.from_numpy(self.cache_np).cuda()
        self.kv = kv
        i32 = dict(dtype=torch.int32, device="cuda")
        i64 = dict(dtype=torch.int64, device="cuda")
        self.maps = dict(query_start=torch.empty(4, **i32), token_to_req_indices=torch.empty(T, **i32), positions=torch.empty(T, **i64),
                         slot_mapping=torch.empty(T, **i64), kv_slot_mapping=torch.empty(T, **i64), kv_lens=torch.empty(3, **i32))
        self.q_in = torch.randn(T, H, 512, generator=g, device="cuda").bfloat16()
        self.k_in = (2 * torch.randn(T, 512, generator=g, device="cuda")).bfloat16()
        self.k_w = 1 + 0.1 * torch.randn(512, generator=g, device="cuda")
        self.sink = torch.randn(H, generator=g, device="cuda")
        self.cos_sin = torch.empty(128, 64, device="cuda")
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros(T, H, 512, **bf)
        self.part = torch.zeros(2, T, H, 512, **bf)
        self.part_lse = torch.full((2, T, H), -math.inf, device="cuda")
        self.merged, self.out = torch.zeros(T, H, 512, **bf), torch.zeros(T, H, 512, **bf)
        self.lse = torch.zeros(T, H, device="cuda")
        self.scale = 512 ** -0.5
        self.ws = [torch.empty(binding.decode_attention_workspace(H), dtype=torch.uint8, device="cuda") for _ in range(2)]
        # every token attends to its request's compressed entries, as a token's decode does
        self.rows = torch.zeros(T, self.kv_table.shape[1], **i32)
        self.rows_lens = torch.zeros(T, **i32)

    def run(self, stream=None):
        m = self.maps
        binding.build_cos_sin(binding.rope(), 0, self.cos_sin, stream=stream)
        binding.build_slot_maps(self.seq_lens, self.query_lens, self.state_table, BLOCK, self.kv_table, KV_BLOCK, RATIO, stream=stream, **m)
        binding.norm_rope_store(m["positions"], m["slot_mapping"], EPS, self.cos_sin, q=self.q_in, q_out=self.q, k=self.k_in, k_w=self.k_w,
                                k_cache=self.cache, kv_block_size=BLOCK, stream=stream)
        binding.window_attention(self.q, self.cache, BLOCK, self.table, m["token_to_req_indices"], m["positions"], m["slot_mapping"],
                                 WINDOW, self.scale, self.part[0], first=FIRST, lse=self.part_lse[0], sink=self.sink, workspace=self.ws[0],
                                 stream=stream)
        with torch.cuda.stream(stream):
            req = m["token_to_req_indices"].long()
            self.rows.copy_(self.kv_table[req])
            self.rows_lens.copy_(torch.where(m["slot_mapping"] >= 0, (m["positions"] + 1) // RATIO, 0))
        binding.decode_attention(self.q, self.kv_cache, KV_BLOCK, self.rows, self.rows_lens, self.scale, self.part[1], lse=self.part_lse[1],
                                 workspace=self.ws[1], stream=stream)
        binding.merge_attention(self.part, self.part_lse, self.merged, lse=self.lse, stream=stream)
        binding.rotate(self.merged, m["positions"], self.cos_sin, self.out, first_column=448, inverse=True, stream=stream)


def check(s):
    """Each link against its formula in 64 bits, from what the link before stored; the attention and all behind it as one."""
    q, out, lse = (x.double().cpu().numpy() for x in (s.q, s.out, s.lse))
    q_in, k_in, k_w, sink = (x.double().cpu().numpy() for x in (s.q_in, s.k_in, s.k_w, s.sink))
    cache = s.cache.cpu().numpy()
    table, _ = ref.cos_sin(0, 128, width=64)
    t = 0
    for r, (n, new) in enumerate(zip(s.lens, s.new)):
        k = sref.entries(cache, BLOCK, s.table_np[r], n)
        far = sref.entries(s.kv_cache_np, KV_BLOCK, s.kv_table_np[r], n // RATIO)
        for p in range(n - new, n):
            cs = table[p:p + 1]
            want, tol = ref.queries(q_in[t:t + 1], None, EPS, cs, "bf16")
            assert (np.abs(q[t] - want[0]) <= tol[0]).all(), (r, p)
            row = k_in[t] / np.sqrt((k_in[t] * k_in[t]).mean() + EPS) * k_w
            row, mag = (a[0, 0] for a in ref.rotate(row[None, None], cs, 448, "pairs", False))
            top = np.repeat(np.abs(row[:448]).reshape(7, 64).max(1), 64)
            # half a step of e4m3, of its smallest binade (2^-10 of the scale, which is at most top / 224) at least; 2^-7 for
            # what the row is off before it
            assert (np.abs(k[p, :448] - row[:448]) <= np.abs(row[:448]) * (2.0 ** -4 + 2.0 ** -7) + top / 224 * 2.0 ** -10).all(), (r, p)
            assert (np.abs(k[p, 448:] - row[448:]) <= sref.HALF_BF16 * np.abs(row[448:]) + 2.0 ** -18 * mag[448:]).all(), (r, p)
            near = k[ref.seen(p, WINDOW, FIRST, 1 << 20)]
            a, la, ta, da = sref.attention(q[t], near, s.scale, sink)
            b, lb, tb, db = sref.attention(q[t], far[:(p + 1) // RATIO], s.scale)
            want, l, mag = sref.merge(np.stack([a, b]), np.stack([la, lb]))
            # a part's weight is off by a factor of at most exp(+-2d), the parts by ta and tb; the merge rounds its sums and to bf16
            d = np.maximum(da, db)[:, None]
            tol = np.maximum(ta, tb) + (np.expm1(2 * d) + 2.0 ** -20) * mag
            tol = tol + sref.HALF_BF16 * (np.abs(want) + tol)
            want, turned = ref.rotate(want[None], cs, 448, "pairs", True)
            _, tol = ref.rotate(tol[None], cs, 448, "pairs", True)
            tol = tol + 2.0 ** -20 * turned
            tol = (tol + sref.HALF_BF16 * (np.abs(want) + tol))[0]
            assert (np.abs(out[t] - want[0]) <= tol).all(), (r, p, np.max(np.abs(out[t] - want[0]) / tol))
            assert (np.abs(lse[t] - l) <= d[:, 0] + 2.0 ** -20 * (1 + np.abs(l))).all(), (r, p)
            t += 1
    assert (q[t:] == 0).all()  # the padded rows were left as they were


def test_step_eager_and_from_a_graph():
    s = Step()
    s.run()
    torch.cuda.synchronize()
    assert binding.device_errors() == 0
    check(s)
    want = [x.clone() for x in (s.out, s.lse, s.cache, s.q)]
    stream = torch.cuda.Stream()
    binding.reserve_workspace(64, stream)
    again = Step()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            again.run(stream)
    for _ in range(3):
        again.out.zero_()
        again.q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (again.out, again.lse, again.cache, again.q)):
            assert torch.equal(a, b)
    assert binding.device_errors(stream) == 0
    binding.release_stream(stream)


def test_steps_on_two_streams_at_once():
    """Two steps in flight, each with its own tensors and workspaces: as if each were alone."""
    alone = []
    for seed in (1, 2):
        s = Step(seed)
        s.run()
        torch.cuda.synchronize()
        alone.append([x.clone() for x in (s.out, s.lse, s.cache)])
    steps, streams = [Step(1), Step(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream in zip(steps, streams):
            s.run(stream)
    torch.cuda.synchronize()
    for s, stream, want in zip(steps, streams, alone):
        for a, b in zip(want, (s.out, s.lse, s.cache)):
            assert torch.equal(a, b)
        assert binding.device_errors(stream) == 0
        binding.release_stream(stream)
