"""The binding of the operators around the compressor without a GPU: which stream its own allocations belong to."""
import contextlib

import pytest

from deepseek_v4_sparse_c128_gb300 import binding, build


class FakeTensor:
    """As much of a CUDA tensor as the binding looks at."""

    def __init__(self, shape, dtype, index=0):
        import torch
        self.shape, self.dtype = tuple(shape), dtype
        self.device = torch.device("cuda", index)
        self._stride = [1] * len(self.shape)
        for i in range(len(self.shape) - 2, -1, -1):
            self._stride[i] = self._stride[i + 1] * self.shape[i + 1]

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return self._stride[i]

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def data_ptr(self):
        return 1 << 20


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class FakeLibrary:
    """The library's signatures; a call is noted and nothing else, so no address here is ever used."""

    def __init__(self, real, calls):
        self._real, self._calls = real, calls

    def __getattr__(self, name):
        return getattr(self._real, name)

    def __getitem__(self, name):
        return lambda *args: self._calls.append((name, args)) or 0


@pytest.fixture
def cuda(monkeypatch):
    """A current stream and device without CUDA, and what torch.empty was asked for on which stream."""
    import torch
    build.build()
    real = binding.load()
    state = {"stream": FakeStream(11), "device": 0, "empty": [], "calls": []}

    @contextlib.contextmanager
    def on(stream):
        before = state["stream"]
        state["stream"] = before if stream is None else stream
        yield
        state["stream"] = before

    def empty(n, dtype=None, device=None):
        state["empty"].append((n, state["stream"].cuda_stream))
        return FakeTensor([n], dtype)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: FakeStream(handle or 99))  # 0: one out of torch's pool
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state["stream"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["device"])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(binding, "decode_attention_workspace", lambda heads: 1000 * heads)
    monkeypatch.setattr(binding, "lib", lambda: FakeLibrary(real, state["calls"]))
    return state


def _decode_args():
    import torch
    return (FakeTensor([3, 5, 512], torch.bfloat16), FakeTensor([4, 2, 584], torch.uint8), 2,
            FakeTensor([3, 9], torch.int32), FakeTensor([3], torch.int32), 0.1, FakeTensor([3, 5, 512], torch.bfloat16))


@pytest.mark.parametrize("stream,owner", [(None, 11), (FakeStream(22), 22), (33, 33), (0, 0), (FakeStream(0), 0)])
def test_own_workspace_belongs_to_the_stream_of_the_call(cuda, stream, owner):
    """torch's allocator orders a block's uses on the stream it was allocated on: another stream's kernel would write into
    memory that queued work still uses, and its own block could be handed out again under it."""
    op = binding.PreparedOp("decode_attention", *_decode_args(), stream=stream)
    op()
    assert cuda["empty"] == [(5000, owner)] and (cuda["calls"][0][1][-1].value or 0) == owner
    cuda["empty"].clear()
    binding.decode_attention(*_decode_args(), stream=stream)
    assert cuda["empty"] == [(5000, owner)]
    assert cuda["stream"].cuda_stream == 11


def test_numbers_that_a_c_integer_does_not_hold_are_refused(cuda):
    """They would reach the library cut to 32 or 64 bits, or to a whole number, as another ratio or block size."""
    import torch
    i32 = lambda *s: FakeTensor(s, torch.int32)
    i64 = lambda *s: FakeTensor(s, torch.int64)
    extend = lambda ratio, block: binding.extend_block_tables(i32(5), i32(5), i32(5, 9), i32(40), i64(1), ratio, block)
    maps = lambda sb, kb, ratio: binding.build_slot_maps(i32(5), i32(5), i32(5, 9), sb, i32(5, 9), kb, ratio, i32(6), i32(7), i64(7),
                                                         i64(7), i64(7), i32(5))
    for ratio, block in [((1 << 32) + 4, 8), (4, (1 << 64) + 8), (4, 8.5), (4.5, 8), (-(1 << 31) - 1, 8)]:
        with pytest.raises(ValueError, match="whole number"):
            extend(ratio, block)
    for sb, kb, ratio in [((1 << 64) + 8, 64, 128), (8, 63.5, 128), (8, 64, (1 << 32) + 128)]:
        with pytest.raises(ValueError, match="whole number"):
            maps(sb, kb, ratio)
    a = list(_decode_args())
    a[2] = (1 << 64) + 2
    with pytest.raises(ValueError, match="whole number"):
        binding.decode_attention(*a)
    assert cuda["calls"] == []
    extend(4, 8.0), maps(8, 64, 128)
    assert [c[0] for c in cuda["calls"]] == ["c128_extend_block_tables", "c128_build_slot_maps"]
    assert [x.value for x in cuda["calls"][0][1][5:7]] == [4, 8]
