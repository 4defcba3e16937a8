"""c128_norm_rope_store on the GPU: queries against a reference in 64 bits, entries byte by byte against the oracle's
epilogue of the same row."""
import numpy as np
import pytest
import torch

import oracle
import step_ref as ref
from deepseek_v4_sparse_c128_gb300 import binding
from test_gpu_step_rotary import KINDS, within

pytestmark = pytest.mark.gpu
EPS = 1e-6


def expected_cache(cache, block, slots, rows, w, eps, cs):
    """The cache's bytes once the rows that have a slot are stored; w may be None."""
    flat = cache.reshape(cache.shape[0], -1)
    w = np.ones(512, np.float32) if w is None else w
    for slot, row, angles in zip(slots, rows, cs):
        if slot < 0:
            continue
        b, off = divmod(int(slot), block)
        tok, sc = oracle.epilogue(np.ascontiguousarray(row), w, eps, np.ascontiguousarray(angles))
        flat[b, off * 576:off * 576 + 576] = tok
        flat[b, block * 576 + off * 8:block * 576 + off * 8 + 8] = sc
    return cache


def inputs(seed, T, H, block, kind, width=584, positions=400):
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(rng.standard_normal((T, H, 512)) * np.exp(rng.standard_normal((1, H, 1)))).to(KINDS[kind])
    k = torch.from_numpy(3 * rng.standard_normal((T, 512))).to(KINDS[kind])
    blocks = T // block + 2
    cache = rng.integers(0, 256, (blocks, block, width), dtype=np.uint8)
    slots = rng.permutation(blocks * block)[:T].astype(np.int64)
    pos = rng.integers(0, positions, T)
    if T > 3:
        slots[T // 2], pos[T // 3] = -1, -5
    angle = rng.uniform(0, 6.3, (positions, 32))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    w = (1 + 0.1 * rng.standard_normal((2, 512))).astype(np.float32)
    return q, k, cache, slots, pos, cs, w


@pytest.mark.parametrize("kind,out_kind", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("T,H,block,width,weights", [(1, 1, 1, 584, False), (1, 64, 64, 584, True), (5, 33, 2, 592, True),
                                                     (40, 7, 3, 584, False), (130, 128, 64, 584, True), (301, 2, 16, 584, False)])
def test_norm_rope_store(T, H, block, width, weights, kind, out_kind):
    q, k, cache, slots, pos, cs, w = inputs(T + H, T, H, block, kind, width)
    kc = torch.from_numpy(cache).cuda()
    before = torch.full((T, H, 512), 3.0, dtype=KINDS[out_kind], device="cuda")
    out = before.clone()
    dev = [torch.from_numpy(a).cuda() for a in (pos, slots, cs, w)]
    binding.norm_rope_store(dev[0], dev[1], EPS, dev[2], q=q.cuda(), q_w=dev[3][0] if weights else None, q_out=out, k=k.cuda(),
                            k_w=dev[3][1] if weights else None, k_cache=kc, kv_block_size=block)
    live = (slots >= 0) & (pos >= 0)
    angles = cs[np.maximum(pos, 0)]
    want, tol = ref.queries(q.double().numpy(), w[0].astype(np.float64) if weights else None, EPS, angles.astype(np.float64), out_kind)
    assert torch.equal(out[~live], before[~live])
    within(out[live], want[live], tol[live])
    expected_cache(cache, block, np.where(live, slots, -1), k.float().numpy(), w[1] if weights else None, EPS, angles)
    assert np.array_equal(kc.cpu().numpy(), cache)
    assert binding.device_errors() == 0


def test_queries_or_keys_alone_and_in_place():
    q, k, cache, slots, pos, cs, w = inputs(5, 37, 9, 4, "bf16")
    dev = [torch.from_numpy(a).cuda() for a in (pos, slots, cs, w)]
    qd, kd, kc = q.cuda(), k.cuda(), torch.from_numpy(cache).cuda()
    both, kc2 = torch.zeros_like(qd), kc.clone()
    binding.norm_rope_store(dev[0], dev[1], EPS, dev[2], q=qd, q_out=both, k=kd, k_w=dev[3][1], k_cache=kc2, kv_block_size=4)
    binding.norm_rope_store(dev[0], dev[1], EPS, dev[2], k=kd, k_w=dev[3][1], k_cache=kc, kv_block_size=4)
    assert torch.equal(kc, kc2)
    live = ((dev[0] >= 0) & (dev[1] >= 0))
    place = qd.clone()
    binding.norm_rope_store(dev[0], dev[1], EPS, dev[2], q=place)
    assert torch.equal(place[live], both[live]) and torch.equal(place[~live], qd[~live])
    # heads first in memory, rows apart; a key with padded rows; a table whose rows start anywhere
    apart = torch.zeros(9, 40, 520, dtype=torch.bfloat16, device="cuda")[:, 3:, 8:].transpose(0, 1)
    wide = torch.zeros(37, 600, dtype=torch.bfloat16, device="cuda")[:, 8:520].copy_(kd)
    table = torch.zeros(400, 67, device="cuda")[:, 3:].copy_(dev[2])
    kc.copy_(torch.from_numpy(cache))
    binding.norm_rope_store(dev[0], dev[1], EPS, table, q=qd, q_out=apart, k=wide, k_w=dev[3][1], k_cache=kc, kv_block_size=4)
    assert torch.equal(apart[live], both[live]) and torch.equal(kc, kc2)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_rows_that_are_not_ordinary(kind):
    """Zeros, one value, values far apart (the mean's slow path), near the type's ends, infinities and NaN: entries byte
    by byte; queries by the formula where it is finite. (The oracle's epilogue is for finite rows: an infinity times the
    root of 1 / infinity, and every value of a row with NaN, is NaN.)"""
    T = 10
    q, k, cache, slots, pos, cs, w = inputs(9, T, 1, 2, kind)
    slots, pos = np.arange(T), np.arange(T)
    k[0] = 0
    k[1] = 0
    k[1, 450] = 4
    k[2] = torch.where(torch.arange(512) % 2 == 0, 1e15, 1e-15).to(KINDS[kind])
    k[3] *= 1e-30
    k[4] *= 1e15
    k[5] *= 1e30
    k[6, 7] = float("inf")
    k[7, 500] = float("nan")
    k[8] = 2.0 ** -126
    k[9, ::2] = -0.0
    q = k[:, None, :].clone()
    kc, out = torch.from_numpy(cache).cuda(), torch.zeros_like(q, device="cuda")
    dev = [torch.from_numpy(a).cuda() for a in (pos, slots, cs, w)]
    binding.norm_rope_store(dev[0], dev[1], EPS, dev[2], q=q.cuda(), q_out=out, k=k.cuda(), k_w=dev[3][1], k_cache=kc, kv_block_size=2)
    expected_cache(cache, 2, slots, k.float().numpy(), w[1], EPS, cs[pos])
    got = kc.cpu().numpy()
    for t in range(T):
        b, off = divmod(t, 2)
        g, e = (a.reshape(a.shape[0], -1)[b] for a in (got, cache))
        if t == 7:
            rec = g[off * 576:off * 576 + 576]
            assert (rec[:448] & 0x7f == 0x7f).all() and np.isnan((rec[448:].view(np.uint16).astype(np.uint32) << 16).view(np.float32)).all()
            continue
        if t == 6:
            assert g[off * 576 + 7] & 0x7f == 0x7f
            e[off * 576 + 7] = g[off * 576 + 7]
        assert np.array_equal(g[off * 576:off * 576 + 576], e[off * 576:off * 576 + 576]), t
        assert np.array_equal(g[2 * 576 + off * 8:][:8], e[2 * 576 + off * 8:][:8]), t
    want, tol = ref.queries(q.double().numpy(), None, EPS, cs[pos].astype(np.float64), kind)
    # squares below 2^-126 may count as 0 in fp32; beside eps that is nothing
    for t in (0, 1, 2, 3, 4, 8, 9):
        within(out[t], want[t], tol[t] + 1e-30)
    assert torch.isnan(out[7]).all()


def test_reports_and_skips():
    q, k, cache, slots, pos, cs, w = inputs(11, 6, 3, 2, "bf16")
    kc = torch.from_numpy(cache).cuda()
    cs_d = torch.from_numpy(cs).cuda()
    out = torch.full((6, 3, 512), 2.0, dtype=torch.bfloat16, device="cuda")
    pos, slots = np.array([0, 400, 1, 1 << 40, -1, 2]), np.array([0, 1, kc.shape[0] * 2, 3, 4, -(1 << 50)])
    dev = [torch.from_numpy(a).cuda() for a in (pos, slots)]
    binding.norm_rope_store(*dev, EPS, cs_d, q=q.cuda(), q_out=out, k=k.cuda(), k_cache=kc, kv_block_size=2)
    assert binding.device_errors() == 8 | 16
    assert (out[1:] == 2).all() and not (out[0] == 2).all()
    expected_cache(cache, 2, np.where(np.arange(6) == 0, slots, -1), k.float().numpy(), None, EPS, cs[np.clip(pos, 0, 399)])
    assert np.array_equal(kc.cpu().numpy(), cache)
    binding.norm_rope_store(*dev, EPS, cs_d, q=q.cuda(), q_out=out)  # without keys a slot is only a sign
    assert binding.device_errors() == 8
    assert not (out[2] == 2).all()
