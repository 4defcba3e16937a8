"""Rows and blocks whose offsets pass 32 bits, in bytes and in elements: the results of compact tensors, bit for bit."""
import numpy as np
import pytest
import torch

from deepseek_v4_sparse_c128_gb300 import binding

pytestmark = pytest.mark.gpu
T, H, BLOCK, BLOCKS = 5, 3, 16, 3


@pytest.fixture(scope="module")
def room():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    yield torch.zeros(24 << 30, dtype=torch.uint8, device="cuda")
    torch.cuda.empty_cache()


def rows(room, shape, stride_t, kind):
    """[T, ..] with `stride_t` elements from a token to the next."""
    inner = [int(np.prod(shape[i + 1:])) for i in range(1, len(shape))]
    return room.view(kind).as_strided(shape, (stride_t, *inner))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("layout", [binding.ROPE_PAIRS, binding.ROPE_HALVES], ids=["pairs", "halves"])
def test_rotate(room, kind, layout):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, 512, generator=g, device="cuda").to(kind)
    cs = torch.empty(8, 64, device="cuda")
    binding.build_cos_sin(binding.rope(), 0, cs)
    pos = torch.arange(T, device="cuda")
    want, stride = torch.empty_like(x), (1 << 30) + 8   # the fifth token's is past 2^32 elements
    binding.rotate(x, pos, cs, want, first_column=448, layout=layout)
    far = rows(room, x.shape, stride, kind)
    far.copy_(x)
    binding.rotate(far, pos, cs, far, first_column=448, layout=layout)
    assert torch.equal(far, want)
    binding.rotate(x, pos, cs, far, first_column=448, layout=layout, inverse=True)
    binding.rotate(x, pos, cs, want, first_column=448, layout=layout, inverse=True)
    assert torch.equal(far, want) and binding.device_errors() == 0


def test_table(room):
    cs = torch.empty(T, 64, device="cuda")
    binding.build_cos_sin(binding.rope(), (1 << 32) - T, cs)
    far = rows(room, cs.shape, (1 << 30) + 4, torch.float32)
    binding.build_cos_sin(binding.rope(), (1 << 32) - T, far)
    assert torch.equal(far, cs)


@pytest.mark.parametrize("window", [20, 300], ids=["short", "long"])
def test_queries_keys_and_attention(room, window):
    g = torch.Generator(device="cuda").manual_seed(2)
    cs = torch.empty(64, 64, device="cuda")
    binding.build_cos_sin(binding.rope(), 0, cs)
    n = BLOCK * BLOCKS
    k = torch.randn(n, 512, generator=g, device="cuda").bfloat16()
    q = torch.randn(T, H, 512, generator=g, device="cuda").bfloat16()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, device="cuda")
    slots = table[0, pos // BLOCK].long() * BLOCK + pos % BLOCK
    req = torch.zeros(T, dtype=torch.int32, device="cuda")
    results = []
    block_bytes = BLOCK * 584
    for far in (False, True):
        # blocks 5 GB apart, and q and out in the room between them, 4 GB from a token to the next
        cache = room.as_strided((BLOCKS, BLOCK, 584), ((5 << 30) if far else block_bytes, 584, 1))
        cache.zero_()
        binding.norm_rope_store(pos, slots, 1e-6, cs, k=k, k_cache=cache, kv_block_size=BLOCK)
        base = room[1 << 20:].view(torch.bfloat16)
        stride = (1 << 31) + 512 if far else 2 * H * 512
        q2 = base.as_strided((T, H, 512), (stride, 512, 1))
        out = base[H * 512:].as_strided((T, H, 512), (stride, 512, 1))
        binding.norm_rope_store(pos[-T:], slots[-T:], 1e-6, cs, q=q, q_out=q2)
        lse = torch.empty(T, H, device="cuda")
        binding.window_attention(q2, cache, BLOCK, table, req, pos[-T:], slots[-T:], window, 512 ** -0.5, out, first=2, lse=lse)
        results.append([x.clone() for x in (cache, q2, out, lse)])
        assert binding.device_errors() == 0
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert bool(results[0][2].any())
