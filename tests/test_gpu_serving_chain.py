"""The operators around the compressor as a serving loop uses them: block tables grow, per-token arrays are made from
them, the compressor stores the windows that end, and the new tokens attend to the compressed cache and to a window
of recent entries, merged. Every step against plain references; the whole also from a captured graph."""
import numpy as np
import pytest

import oracle
from deepseek_v4_sparse_c128_gb300 import inputs
from gpu_util import comp_close
from serving_ref import HEAD, attention, cdiv, entries, make_cache, make_tables, slot_maps

pytestmark = pytest.mark.gpu

RATIO, STATE_BLOCK, KV_BLOCK = 128, 8, 2


@pytest.fixture(scope="module")
def binding():
    from deepseek_v4_sparse_c128_gb300 import binding as b
    from deepseek_v4_sparse_c128_gb300 import build
    build.build()
    b.load()
    oracle.build()
    b.device_errors(clear=True)
    return b


class Server:
    """The device state of a small server; `step` advances it by one call of each operator."""

    def __init__(self, binding, rng, requests, longest, heads, stream=None):
        import torch
        dev = "cuda"
        self.b, self.heads, self.requests = binding, heads, requests
        i32, i64 = torch.int32, torch.int64
        self.state_blocks, self.kv_blocks = requests * cdiv(longest, STATE_BLOCK), requests * cdiv(longest // RATIO, KV_BLOCK) + 1
        z = lambda *s, dtype=i32: torch.zeros(*s, dtype=dtype, device=dev)
        self.lens, self.new = z(requests), z(requests)
        self.state_held, self.kv_held, self.state_taken, self.kv_taken = z(requests), z(requests), z(1, dtype=i64), z(1, dtype=i64)
        self.state_table = torch.full((requests, cdiv(longest, STATE_BLOCK)), -1, dtype=i32, device=dev)
        self.kv_table = torch.full((requests, cdiv(longest // RATIO, KV_BLOCK) + 1), -1, dtype=i32, device=dev)
        self.state_free = torch.from_numpy(rng.permutation(self.state_blocks).astype(np.int32)).to(dev)
        self.kv_free = torch.from_numpy(rng.permutation(self.kv_blocks).astype(np.int32)).to(dev)
        self.tokens = requests * 300
        self.maps = {"query_start": z(requests + 1), "token_to_req_indices": z(self.tokens), "positions": z(self.tokens, dtype=i64),
                     "slot_mapping": z(self.tokens, dtype=i64), "kv_slot_mapping": z(self.tokens, dtype=i64), "kv_lens": z(requests)}
        self.state = torch.from_numpy(rng.standard_normal((self.state_blocks, 8, 1024)).astype(np.float32)).to(dev)
        self.rms_w = torch.from_numpy((1 + 0.1 * rng.standard_normal(HEAD)).astype(np.float32)).to(dev)
        self.cos_sin = torch.from_numpy(inputs._cos_sin_cache(longest)).to(dev)
        self.cache = torch.zeros(self.kv_blocks, KV_BLOCK, 584, dtype=torch.uint8, device=dev)
        self.comp = torch.zeros(self.tokens, HEAD, device=dev)
        # the window of recent entries: another cache of the same layout, one block of 64 per request
        self.window = torch.from_numpy(make_cache(rng, requests, 64)).to(dev)
        self.window_table = torch.arange(requests, dtype=i32, device=dev)[:, None].contiguous()
        self.window_lens = torch.from_numpy(rng.integers(1, 65, requests).astype(np.int32)).to(dev)
        self.q = torch.from_numpy(rng.standard_normal((requests, heads, HEAD)).astype(np.float32)).to(torch.bfloat16).to(dev)
        self.sink = torch.from_numpy(rng.standard_normal(heads).astype(np.float32)).to(dev)
        self.part = torch.zeros(2, requests, heads, HEAD, device=dev)
        self.part_lse = torch.zeros(2, requests, heads, device=dev)
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(requests, heads, device=dev)
        self.scale = HEAD ** -0.5
        P = lambda op, *a, **k: binding.PreparedOp(op, *a, stream=stream, **k)
        m = self.maps
        self.calls = [
            P("extend_block_tables", self.lens, self.state_held, self.state_table, self.state_free, self.state_taken, 1, STATE_BLOCK),
            P("extend_block_tables", self.lens, self.kv_held, self.kv_table, self.kv_free, self.kv_taken, RATIO, KV_BLOCK),
            P("build_slot_maps", self.lens, self.new, self.state_table, STATE_BLOCK, self.kv_table, KV_BLOCK, RATIO, **m),
            binding.PreparedCall(m["token_to_req_indices"], m["positions"], m["slot_mapping"], self.state_table, self.state,
                                 self.rms_w, 1e-6, self.cos_sin, self.cache, m["kv_slot_mapping"], KV_BLOCK, stream=stream,
                                 comp_out=self.comp),
            P("decode_attention", self.q, self.cache, KV_BLOCK, self.kv_table, m["kv_lens"], self.scale, self.part[0],
              lse=self.part_lse[0], sink=self.sink),
            P("decode_attention", self.q, self.window, 64, self.window_table, self.window_lens, self.scale, self.part[1],
              lse=self.part_lse[1]),
            P("merge_attention", self.part, self.part_lse, self.out, lse=self.lse),
        ]

    def step(self):
        for call in self.calls:
            call()

    def check(self):
        """This step's results against the references."""
        n = lambda t: t.cpu().numpy()
        lens, new = n(self.lens), n(self.new)
        st, kt = n(self.state_table), n(self.kv_table)
        # every request holds the blocks its length needs, each block once
        for table, held, need in ((st, n(self.state_held), [cdiv(int(x), STATE_BLOCK) for x in lens]),
                                  (kt, n(self.kv_held), [cdiv(int(x) // RATIO, KV_BLOCK) for x in lens])):
            assert list(held) == need
            used = np.concatenate([table[r, :need[r]] for r in range(len(need))])
            assert (used >= 0).all() and len(set(used.tolist())) == len(used)
            assert all((table[r, need[r]:] == -1).all() for r in range(len(need)))
        want, bits = slot_maps(lens, new, st, STATE_BLOCK, kt, KV_BLOCK, RATIO, self.tokens)
        assert bits == 0
        for k, v in want.items():
            assert np.array_equal(n(self.maps[k]), v), k
        # the windows that ended this step: the compressed vectors, and the cache bytes they give
        cache, state, comp = n(self.cache), n(self.state), n(self.comp)
        ends = np.nonzero((want["slot_mapping"] >= 0) & (want["kv_slot_mapping"] >= 0))[0]
        p = inputs.Problem(name="step", token_to_req=want["token_to_req_indices"], positions=want["positions"],
                           slot_mapping=want["slot_mapping"], block_table=st, state=state, rms_w=n(self.rms_w), eps=1e-6,
                           cos_sin=n(self.cos_sin), k_cache=np.zeros_like(cache), kv_slot_mapping=want["kv_slot_mapping"],
                           kv_block_size=KV_BLOCK)
        ref = np.zeros_like(comp)
        assert oracle.forward(p, k_cache=p.k_cache.copy(), comp_out=ref) == 0
        ok, _, worst = comp_close(comp[ends], ref[ends])
        assert ok, worst
        for t in ends[:40]:
            pos, s = int(want["positions"][t]), int(want["kv_slot_mapping"][t])
            rec, sc = oracle.epilogue(comp[t], p.rms_w, 1e-6, p.cos_sin[(pos // RATIO) * RATIO])
            flat = cache[s // KV_BLOCK].reshape(-1)
            assert np.array_equal(flat[(s % KV_BLOCK) * 576:][:576], rec)
            assert np.array_equal(flat[KV_BLOCK * 576 + (s % KV_BLOCK) * 8:][:8], sc)
        # attention over both caches at once
        q, window, out, lse = n(self.q.double()), n(self.window), n(self.out.double()), n(self.lse.double())
        for r in range(self.requests):
            k = np.concatenate([entries(cache, KV_BLOCK, kt[r], int(lens[r]) // RATIO),
                                entries(window, 64, [r], int(n(self.window_lens)[r]))])
            want_out, want_lse, tol, tol_lse = attention(q[r], k, self.scale, n(self.sink).astype(np.float64))
            # the merge adds a weight's exp and the sums of two parts in fp32, below 2^-16 of the magnitudes
            tol = tol + 2.0 ** -16 * np.abs(k).max(initial=0)
            assert (np.abs(out[r] - want_out) <= tol).all(), r
            assert (np.abs(lse[r] - want_lse) <= tol_lse + 2.0 ** -16).all(), r


def test_serving_steps(binding):
    """A prefill of ragged prompts, then decode steps and another chunk of tokens."""
    import torch
    rng = np.random.default_rng(31)
    s = Server(binding, rng, 9, 1500, 20)
    for new in ([300, 0, 128, 127, 1, 255, 256, 299, 64], [1] * 9, [0, 1, 1, 129, 127, 0, 1, 300, 200], [1] * 9):
        s.new.copy_(torch.tensor(new, dtype=torch.int32))
        s.lens += s.new
        s.step()
        assert binding.device_errors(clear=True) == 0
        s.check()


def test_serving_steps_from_a_graph(binding):
    """The same loop captured once and replayed, lengths changing on the device."""
    import torch
    rng = np.random.default_rng(32)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s = Server(binding, rng, 5, 1200, 64, stream=stream)
        binding.reserve_workspace(s.tokens, stream=stream)
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s.lens += s.new
            s.step()
        for new in ([300, 200, 0, 128, 5], [1] * 5, [127, 55, 256, 1, 0]):
            s.new.copy_(torch.tensor(new, dtype=torch.int32))
            g.replay()
            stream.synchronize()
            assert binding.device_errors(stream, clear=True) == 0
            s.check()
    binding.release_stream(stream)
