"""c128_build_cos_sin and c128_rotate on the GPU against references in 64 bits."""
import numpy as np
import pytest
import torch

import step_ref as ref
from deepseek_v4_sparse_c128_gb300 import binding

pytestmark = pytest.mark.gpu
KINDS = {"bf16": torch.bfloat16, "fp32": torch.float32}


def within(got, want, tol):
    got = got.double().cpu().numpy()
    worst = np.abs(got - want) / np.maximum(tol, 1e-300)
    assert (np.abs(got - want) <= tol).all(), f"worst {worst.max():.3g} of the tolerance"


@pytest.mark.parametrize("width,rows,first", [(2, 1, 0), (2, 1000, 7), (64, 1, 131071), (64, 5000, 0), (96, 333, 1 << 20),
                                              (128, 257, (1 << 32) - 257), (510, 19, 5), (512, 70, 0)])
@pytest.mark.parametrize("rope", [
    dict(), dict(theta=500000.0, scaling="linear", factor=8.0), dict(scaling="yarn", factor=16.0, magnitude=1.2772588722239782),
    dict(theta=1.5, scaling="yarn", factor=0.5, original_positions=300, beta_fast=2.0, beta_slow=1.0),
    dict(scaling="yarn", factor=40.0, original_positions=4, magnitude=-2.0)])
def test_table(width, rows, first, rope):
    table = torch.full((rows, width + 3), 7.0, device="cuda")
    binding.build_cos_sin(binding.rope(**rope), first, table[:, :width])
    want, tol = ref.cos_sin(first, rows, width=width, **rope)
    within(table[:, :width], want, tol)
    assert (table[:, width:] == 7).all()


def test_table_long():
    """More rows than threads on the GPU: the angles go on by addition."""
    table = torch.empty(300001, 64, device="cuda")
    binding.build_cos_sin(binding.rope(), 12345, table)
    at = torch.arange(0, 300001, 101)
    want, tol = ref.cos_sin(12345, 300001, width=64)
    within(table[at.cuda()], want[at.numpy()], tol[at.numpy()])


def table_for(rng, rows, width, odd=0):
    """A table of random angles; odd: its rows do not start on 16 bytes."""
    angle = rng.uniform(0, 6.3, (rows, width // 2))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    whole = torch.zeros(rows, width + odd, device="cuda")
    whole[:, odd:] = torch.from_numpy(cs).cuda()
    return whole[:, odd:], cs.astype(np.float64)


SHAPES = [  # tokens, heads, width, first, turned
    (1, 1, 2, 0, 2), (1, 64, 512, 448, 64), (7, 3, 512, 448, 64), (5, 33, 128, 0, 64), (3, 2, 97, 5, 34), (300, 1, 64, 0, 64),
    (1000, 2, 8, 0, 8), (2, 40, 192, 128, 64), (17, 5, 96, 32, 32), (4, 3, 136, 8, 112), (2, 2, 520, 4, 512),
]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rotate(shape, layout, kind):
    T, H, D, first, turned = shape
    rng = np.random.default_rng(sum(shape) + len(layout))
    for inverse in (False, True):
        for where in ("out", "place", "strided"):
            x = torch.from_numpy(rng.standard_normal((T, H, D))).to(KINDS[kind]).cuda()
            cs, cs64 = table_for(rng, 50, turned, odd=1 if where == "strided" else 0)
            pos = rng.integers(0, 50, T)
            if T > 2:
                pos[T // 2] = -1
            positions = torch.from_numpy(pos).cuda()
            want, mag = ref.rotate(x.double().cpu().numpy(), cs64[np.maximum(pos, 0)], first, layout, inverse)
            tol = ref.rotate_tolerance(want, mag, kind)
            before = torch.full((T, H, D), 3.0, dtype=KINDS[kind], device="cuda")
            if where == "strided":  # heads first in memory, odd distances
                x = torch.zeros(H, T, D + 1, dtype=KINDS[kind], device="cuda")[..., 1:].transpose(0, 1).copy_(x)
                out = torch.zeros(T, H + 1, D + 3, dtype=KINDS[kind], device="cuda")[:, 1:, 3:].copy_(before)
            elif where == "place":
                out, before = x, x.clone()
            else:
                out = before.clone()
            layouts = {"pairs": binding.ROPE_PAIRS, "halves": binding.ROPE_HALVES}
            binding.rotate(x, positions, cs, None if where == "place" else out, first_column=first, layout=layouts[layout],
                           inverse=inverse)
            skipped = pos < 0
            assert torch.equal(out[skipped], before[skipped])
            within(out[~skipped], want[~skipped], tol[~skipped])
            if where == "place":  # columns that do not turn keep their bits
                rest = [c for c in range(D) if not first <= c < first + turned]
                assert torch.equal(out[..., rest], before[..., rest])
    assert binding.device_errors() == 0


def test_rotate_back():
    """There and back: two roundings of bf16 and four of fp32 apart."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(40, 8, 512, generator=g, device="cuda")
    positions = torch.randint(1 << 20, (40,), generator=g, device="cuda")
    cs = torch.empty(1 << 20, 64, device="cuda")
    binding.build_cos_sin(binding.rope(), 0, cs)
    there, back = torch.empty_like(x), torch.empty_like(x)
    binding.rotate(x, positions, cs, there, first_column=448)
    binding.rotate(there, positions, cs, back, first_column=448, inverse=True)
    # cos^2 + sin^2 is 1 up to 2^-22 (each within 2^-23 of its value); the sums of either turn are off by 2^-23 of their magnitudes
    mag = x[..., 448:].abs().unflatten(-1, (32, 2)).sum(-1, keepdim=True).expand(-1, -1, -1, 2).flatten(-2)
    assert ((back - x)[..., 448:].abs() <= 2.0 ** -20 * mag).all()
    assert torch.equal(back[..., :448], x[..., :448])


def test_rotate_reports_positions_behind_the_table():
    x = torch.randn(4, 2, 64, device="cuda")
    cs = torch.ones(10, 64, device="cuda")
    out = torch.full_like(x, 5.0)
    binding.rotate(x, torch.tensor([3, 10, -1, 1 << 40], device="cuda"), cs, out)
    assert binding.device_errors() == 8
    assert (out[1:] == 5).all() and not (out[0] == 5).any()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_rotate_passes_what_is_not_finite(kind):
    x = torch.zeros(1, 3, 80, dtype=KINDS[kind], device="cuda")
    x[0, 0, 70], x[0, 1, 3], x[0, 2, 0] = float("nan"), float("inf"), float("-inf")
    cs = torch.tensor([[1.0] * 32 + [0.5] * 32], device="cuda")
    out = torch.empty_like(x)
    binding.rotate(x, torch.zeros(1, dtype=torch.int64, device="cuda"), cs, out, layout=binding.ROPE_PAIRS)
    assert torch.isnan(out[0, 0, 70]) and torch.isfinite(out[0, 0, :70]).all()
    assert out[0, 1, 3].item() == float("inf") and out[0, 1, 2].item() == -float("inf")
    assert out[0, 2, 0].item() == -float("inf") and out[0, 2, 1].item() == -float("inf")


def test_rotate_in_a_graph_and_on_a_stream():
    x = torch.randn(9, 4, 512, device="cuda").bfloat16()
    cs = torch.empty(100, 64, device="cuda")
    pos = torch.arange(9, device="cuda") * 11
    out, again = torch.zeros_like(x), torch.zeros_like(x)
    binding.build_cos_sin(binding.rope(), 0, cs)
    binding.rotate(x, pos, cs, out, first_column=448)
    s = torch.cuda.Stream()
    binding.reserve_workspace(1, s)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            cs.zero_()
            binding.build_cos_sin(binding.rope(), 0, cs)
            binding.rotate(x, pos, cs, again, first_column=448)
    for _ in range(3):
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, again)
    binding.release_stream(s)
