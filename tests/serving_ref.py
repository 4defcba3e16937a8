"""Plain references, in 64 bits on the CPU, of the operators around the compressor, and how far their
results may be from them. Written from the contracts in include/c128compress.h."""
import math

import numpy as np
import torch

HEAD, NOPE, GROUP, RECORD, SCALES = 512, 448, 64, 576, 8
HALF_BF16 = 2.0 ** -8     # half a step of bf16, relative to the value
HALF_F32 = 2.0 ** -24


def cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------- tables and maps
def extend(seq_lens, held, table, free, taken, ratio, block):
    """(table, held, taken, error bits) after c128_extend_block_tables, one block at a time."""
    table, held_out, bits, at, stopped = table.copy(), held.copy(), 0, int(taken), False
    if not 0 <= at <= len(free):
        bits, stopped = bits | 128, True
    for r in range(len(seq_lens)):
        n = int(seq_lens[r])
        if n < 0:
            bits, n = bits | 128, 0
        needed = cdiv(n // ratio, block)
        if held[r] < 0:
            bits |= 128
            continue
        if needed <= held[r]:
            continue
        if needed > table.shape[1]:
            bits |= 2
            continue
        if stopped or at + needed - held[r] > len(free):
            bits, stopped = bits | 64, True
            continue
        for j in range(held[r], needed):
            table[r, j] = free[at]
            at += 1
        held_out[r] = needed
    return table, held_out, at, bits


def slot_maps(seq_lens, query_lens, state_table, state_block, kv_table, kv_block, ratio, tokens):
    """The outputs of c128_build_slot_maps as a dict, and the error bits."""
    bits, rows, start = 0, [], [0]

    def slot(table, r, index, block):
        nonlocal bits
        if index // block >= table.shape[1]:
            bits |= 2
            return -1
        if table[r, index // block] < 0:
            bits |= 4
            return -1
        return int(table[r, index // block]) * block + index % block

    lens, new = np.maximum(seq_lens, 0), np.maximum(query_lens, 0)
    if (seq_lens < 0).any() or (query_lens < 0).any() or (new > lens).any() or new.astype(np.int64).sum() > tokens:
        bits |= 128
    for r in range(len(lens)):
        for i in range(new[r]):
            if len(rows) == tokens:
                break
            p = int(lens[r]) - int(new[r]) + i
            s = k = -1
            if p >= 0:
                s = slot(state_table, r, p, state_block)
                if (p + 1) % ratio == 0:
                    k = slot(kv_table, r, p // ratio, kv_block)
            rows.append((r, p, s, k))
        start.append(start[-1] + int(new[r]))
    rows += [(0, 0, -1, -1)] * (tokens - len(rows))
    a = np.array(rows, dtype=np.int64).reshape(tokens, 4)
    return {"query_start": np.array(start, dtype=np.int32), "token_to_req_indices": a[:, 0].astype(np.int32),
            "positions": a[:, 1], "slot_mapping": a[:, 2], "kv_slot_mapping": a[:, 3],
            "kv_lens": (lens // ratio).astype(np.int32)}, bits


# ------------------------------------------------------------------------------------- attention
def e4m3_values():
    """Value of every e4m3 byte from the format: sign, 4 exponent bits of bias 7, 3 mantissa bits, 0x7f NaN."""
    def value(b):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if b & 127 == 127 else math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        return -v if b & 128 else v
    return np.array([value(b) for b in range(256)])


def entries(cache, block, pages, n):
    """Entries 0 .. n-1 of a request with these pages: [n, 512] in 64 bits. Pages outside the cache give NaN rows."""
    out = np.full((n, HEAD), np.nan)
    values = e4m3_values()
    for j in range(n):
        b, off = int(pages[j // block]), j % block
        if not 0 <= b < cache.shape[0]:
            continue
        flat = cache[b].reshape(-1)
        rec = flat[off * RECORD:(off + 1) * RECORD]
        scale = flat[block * RECORD + off * SCALES:][:NOPE // GROUP].astype(np.float64)
        out[j, :NOPE] = values[rec[:NOPE]] * np.repeat(np.exp2(scale - 127), GROUP)
        out[j, NOPE:] = (rec[NOPE:].view(np.uint16).astype(np.uint32) << 16).view(np.float32)
    return out


def attention(q, k, scale, sink=None, out_half=HALF_BF16):
    """(out, lse, tolerance of out, tolerance of lse) of one request: q [H, 512], k [n, 512], sink [H].

    The tolerances: scores add 512 products in fp32, each sum off by at most 2^-23 of the magnitudes (the tensor
    cores cut instead of rounding), so a score is off by d = 2^-14 * scale * sum|q k|, its weight by a factor
    exp(+-d), and so is the sum of weights. A weight is rounded to bf16 (2^-8) and the result to its type. Sums over
    the entries in fp32 and the exponential's own error (2^-22) are taken together as 2^-16."""
    n, heads = k.shape[0], q.shape[0]
    s = scale * (q @ k.T) if n else np.zeros((heads, 0))
    d = 2.0 ** -14 * abs(scale) * (np.abs(q) @ np.abs(k).T).max(1) if n else np.zeros(heads)
    if sink is not None:
        s = np.concatenate([s, sink[:, None]], 1)
        k = np.concatenate([k, np.zeros((1, HEAD))])
    if not s.shape[1]:
        return np.zeros((heads, HEAD)), np.full(heads, -np.inf), np.zeros((heads, HEAD)), np.zeros(heads)
    top = s.max(1)
    lse = top + np.log(np.exp(s - top[:, None]).sum(1))
    p = np.exp(s - lse[:, None])
    out = p @ k
    tol = out_half * np.abs(out) + (p @ np.abs(k)) * (HALF_BF16 + 2 * d + 2.0 ** -16)[:, None]
    return out, lse, tol, d + 2.0 ** -16 + 2.0 ** -22 * np.abs(lse)


def make_cache(rng, num_blocks, block, width=584):
    """A cache of random records as the compressor writes them (values near N(0, 1)), stale bytes where a block is
    wider than its records."""
    n = num_blocks * block
    x = torch.from_numpy(rng.standard_normal((n, HEAD)).astype(np.float32))
    nope = x[:, :NOPE].reshape(n, -1, GROUP)
    e = torch.ceil(torch.log2(nope.abs().amax(-1).clamp_min(1e-4) / 448))
    codes = (nope * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(n, NOPE)
    data = torch.cat([codes, x[:, NOPE:].to(torch.bfloat16).view(torch.uint8)], 1).numpy()
    scales = np.zeros((n, SCALES), np.uint8)
    scales[:, :NOPE // GROUP] = (e + 127).to(torch.uint8).numpy()
    cache = rng.integers(0, 256, (num_blocks, block * width), dtype=np.uint8)
    cache[:, :block * RECORD] = data.reshape(num_blocks, -1)
    cache[:, block * RECORD:block * (RECORD + SCALES)] = scales.reshape(num_blocks, -1)
    return cache.reshape(num_blocks, block, width)


def make_tables(rng, lens, block, num_blocks, columns=None):
    """Distinct random pages for each request, -1 behind them."""
    need = [cdiv(max(0, int(n)), block) for n in lens]
    table = np.full((len(lens), columns or max(1, max(need, default=1))), -1, np.int32)
    pages, at = rng.permutation(num_blocks).astype(np.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = pages[at:at + n]
        at += n
    return table


def merge(part_out, part_lse):
    """(out, lse, sum of weights x |part|) of partial attentions [P, .., 512] and [P, ..] in 64 bits."""
    top = part_lse.max(0)
    shift = np.where(np.isinf(top), 0, top)
    w = np.exp(part_lse - shift)
    total = w.sum(0)
    part = np.where((w > 0)[..., None], part_out, 0)
    inv = np.where(total > 0, 1 / np.where(total > 0, total, 1), 0)
    out = (w[..., None] * part).sum(0) * inv[..., None]
    mag = (w[..., None] * np.abs(part)).sum(0) * inv[..., None]
    with np.errstate(divide="ignore"):
        lse = shift + np.log(total)
    return out, lse, mag
