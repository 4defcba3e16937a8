"""Cases of the operators that stand around the compressor, for timing and comparison.

Four operators, each in a plain form (elementary torch operations) and as the calls of this package:

* ``tables``  block tables grown from request lengths out of a list of free blocks;
* ``maps``    the compressor's per-token arrays (request, position, state slot, cache slot) of one step;
* ``decode``  attention of one new token per request over the paged FP8 cache the compressor writes;
* ``merge``   partial attentions over several caches joined by their log-sum-exp.

A case fixes the sizes and how long the requests are (the set of lengths); the seed draws the values, the order of
the requests and the order of the physical blocks.
"""
import math

import torch

own = False

HEAD, NOPE, GROUP = 512, 448, 64   # head size, its FP8 part, columns per UE8M0 scale
RECORD, SCALES = 576, 8            # bytes of an entry's data and of its scales
STATE_BLOCK = 8                    # tokens per block of the compressor's state cache


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of a busy server: every request one token longer, few of them into a new state block
        {"name": "tables_decode", "op": "tables", "requests": 256, "longest": 8192, "spread": "even", "grow": 1,
         "ratio": 1, "block": 8},
        # long prompts arrive: 16 requests of up to a million tokens get all their state blocks at once
        {"name": "tables_prefill", "op": "tables", "requests": 16, "longest": 1048576, "spread": "even", "grow": 0,
         "ratio": 1, "block": 8},
        # one decode step, arrays padded to the size that the captured graph was made for
        {"name": "maps_decode", "op": "maps", "requests": 200, "longest": 16374, "spread": "even", "query": 1,
         "pad": 56, "ratio": 128, "kv_block": 64},
        # chunked prefill among decodes: ragged numbers of new tokens, some requests with none
        {"name": "maps_mixed", "op": "maps", "requests": 333, "longest": 131072, "spread": "skew", "query": 200,
         "pad": 0, "ratio": 4, "kv_block": 2},
        # whole prompts and parts of prompts, about 200 thousand new tokens
        {"name": "maps_prefill", "op": "maps", "requests": 17, "longest": 32768, "spread": "even", "query": 32768,
         "pad": 0, "ratio": 128, "kv_block": 64},
        # one request at 128 Ki tokens of context (ratio 128): latency counts
        {"name": "decode_one", "op": "decode", "requests": 1, "heads": 64, "longest": 1024, "spread": "full",
         "kv_block": 64, "sink": False},
        # a decode batch at up to 128 Ki tokens of context
        {"name": "decode_batch", "op": "decode", "requests": 64, "heads": 64, "longest": 1024, "spread": "even",
         "kv_block": 64, "sink": True},
        # many short and some empty requests, two entries to a block, an odd number of heads
        {"name": "decode_short", "op": "decode", "requests": 250, "heads": 33, "longest": 300, "spread": "skew",
         "kv_block": 2, "sink": True},
        # few heads on this GPU and a long cache (ratio 4): the cache read is all there is
        {"name": "decode_long", "op": "decode", "requests": 8, "heads": 16, "longest": 65536, "spread": "even",
         "kv_block": 64, "sink": False},
        # 128 heads, up to 1 Mi tokens of context: the products count
        {"name": "decode_wide", "op": "decode", "requests": 48, "heads": 128, "longest": 8192, "spread": "skew",
         "kv_block": 64, "sink": False},
        # window attention joined with compressed attention, one request
        {"name": "merge_one", "op": "merge", "requests": 1, "heads": 64, "parts": 2, "lse": True},
        # a large batch over four partial results
        {"name": "merge_batch", "op": "merge", "requests": 256, "heads": 128, "parts": 4, "lse": True},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "maps", "decode", "decode", "decode", "merge"])
    spread = rng.choice(["full", "even", "skew"])
    if op == "tables":
        requests, ratio, block = _log_uniform(rng, 1, 2048), rng.choice([1, 4, 128]), rng.choice([2, 8, 64])
        longest = _log_uniform(rng, 1, max(1, min(1 << 20, (1 << 24) // requests)))
        return {"op": op, "requests": requests, "longest": longest, "spread": spread,
                "grow": rng.choice([0, 1, rng.randint(1, longest)]), "ratio": ratio, "block": block}
    if op == "maps":
        requests, longest = _log_uniform(rng, 1, 2048), _log_uniform(rng, 1, 1 << 17)
        query = min(longest, _log_uniform(rng, 1, max(1, (1 << 18) // requests)))
        return {"op": op, "requests": requests, "longest": longest, "spread": spread, "query": query,
                "pad": rng.choice([0, rng.randint(1, 300)]), "ratio": rng.choice([4, 128]),
                "kv_block": rng.choice([1, 2, 64])}
    if op == "decode":
        requests, heads = _log_uniform(rng, 1, 256), _log_uniform(rng, 1, 128)
        longest = _log_uniform(rng, 1, max(1, min(65536, (1 << 18) // requests, 12000000 // (requests * heads))))
        return {"op": op, "requests": requests, "heads": heads, "longest": longest, "spread": spread,
                "kv_block": rng.choice([1, 2, 16, 64, 67]), "sink": rng.random() < 0.5}
    return {"op": op, "requests": _log_uniform(rng, 1, 256), "heads": rng.randint(1, 128),
            "parts": rng.randint(1, 4), "lse": rng.random() < 0.5}


def _lengths(n, longest, spread):
    """The n lengths of a case, 0 .. longest: all the longest, evenly spread, or most of them short."""
    if spread == "full":
        return [longest] * n
    if spread == "even":
        return [max(1, longest * (i + 1) // n) for i in range(n)]
    return [int(longest * (i / n) ** 3) for i in range(n - 1)] + [longest]


def _queries(case):
    """New tokens of each request: one in a decode step, else 0 .. query (the longest request has `query`)."""
    lens, query = _lengths(case["requests"], case["longest"], case["spread"]), case["query"]
    if query == 1:
        return [min(1, n) for n in lens]
    return [min(n, query * ((7 * i) % 11) // 10) for i, n in enumerate(lens[:-1])] + [query]


def _cdiv(a, b):
    return -(-a // b)


def _table_lengths(case):
    """(length before, length now) of each request."""
    now = _lengths(case["requests"], case["longest"], case["spread"])
    return [(max(0, n - case["grow"]) if case["grow"] else 0, n) for n in now]


def work(case):
    if case["op"] == "tables":
        blocks = sum(_cdiv(n // case["ratio"], case["block"]) - _cdiv(o // case["ratio"], case["block"])
                     for o, n in _table_lengths(case))
        return {"bytes": 12 * case["requests"] + 8 * blocks + 16, "flops": 0}
    if case["op"] == "maps":
        lens, new = _lengths(case["requests"], case["longest"], case["spread"]), _queries(case)
        tokens = sum(new) + case["pad"]
        read = sum(_cdiv(n, STATE_BLOCK) - (n - q) // STATE_BLOCK for n, q in zip(lens, new))
        span = case["ratio"] * case["kv_block"]
        read += sum(n // span - (n - q) // span for n, q in zip(lens, new))
        return {"bytes": 16 * case["requests"] + 4 + 4 * read + 28 * tokens, "flops": 0}
    rows = case["requests"] * case["heads"]
    if case["op"] == "decode":
        lens = _lengths(case["requests"], case["longest"], case["spread"])
        blocks = sum(_cdiv(n, case["kv_block"]) for n in lens)
        return {"bytes": sum(lens) * (RECORD + SCALES) + 4 * (blocks + case["requests"]) + rows * (4 * HEAD + 4)
                + (4 * case["heads"] if case["sink"] else 0),
                "flops": 4 * HEAD * case["heads"] * sum(lens)}
    return {"bytes": (case["parts"] + 1) * rows * 2 * HEAD + (case["parts"] + case["lse"]) * rows * 4,
            "flops": 2 * case["parts"] * rows * HEAD}


# ------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(values, order=None, dtype=torch.int32):
    v = torch.tensor(values, dtype=dtype, device="cuda")
    return v if order is None else v[order].contiguous()


def _tables(held, columns, g, spare=0):
    """Tables [R, columns] whose first held[r] entries are distinct blocks in random order, -1 after them; the
    blocks left over come back as a list."""
    total = int(held.sum())
    blocks = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(columns, device="cuda")[None, :] < held[:, None]
    table = torch.full(at.shape, -1, dtype=torch.int32, device="cuda")
    table[at] = blocks[:total]
    return table, blocks[total:].contiguous()


def _cache(entries, block, g):
    """A cache of `entries` records (whole blocks): FP8 e4m3 in groups of 64 with UE8M0 scales, the last 64 columns
    bf16. Vectors as they come out of an RMSNorm with a weight near one."""
    x = torch.randn(entries, HEAD, generator=g, device="cuda")
    x *= 1 + 0.1 * torch.randn(HEAD, generator=g, device="cuda")
    nope = x[:, :NOPE].reshape(entries, NOPE // GROUP, GROUP)
    e = torch.ceil(torch.log2(nope.abs().amax(-1).clamp_min(1e-4) / 448))
    codes = (nope * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(entries, NOPE)
    rope = x[:, NOPE:].to(torch.bfloat16).view(torch.uint8)
    data = torch.cat([codes, rope], 1).reshape(entries // block, block * RECORD)
    scales = torch.zeros(entries, SCALES, dtype=torch.uint8, device="cuda")
    scales[:, : NOPE // GROUP] = (e + 127).to(torch.uint8)
    cache = torch.cat([data, scales.reshape(entries // block, block * SCALES)], 1)
    return cache.reshape(entries // block, block, RECORD + SCALES)


def prepare(case, seed):
    g = _generator(seed)
    n, op = case["requests"], case["op"]
    order = torch.randperm(n, generator=g, device="cuda")
    s = {"op": op, "case": case}
    if op == "tables":
        pairs, block = _table_lengths(case), case["block"]
        s["seq_lens"] = _ints([b for _, b in pairs], order)
        need = [_cdiv(b // case["ratio"], block) for _, b in pairs]
        s["held"] = _ints([_cdiv(a // case["ratio"], block) for a, _ in pairs], order)
        s["block_table"], s["free_blocks"] = _tables(s["held"], max(1, max(need)), g, sum(need) + 100 - int(s["held"].sum()))
        s["taken"] = torch.tensor([seed % 100], dtype=torch.int64, device="cuda")
        s["held_out"], s["taken_out"] = torch.empty_like(s["held"]), torch.empty_like(s["taken"])
    elif op == "maps":
        lens, new = _lengths(n, case["longest"], case["spread"]), _queries(case)
        tokens = sum(new) + case["pad"]
        s["seq_lens"], s["query_lens"] = _ints(lens, order), _ints(new, order)
        held = torch.div(s["seq_lens"] + STATE_BLOCK - 1, STATE_BLOCK, rounding_mode="floor")
        s["state_table"], _ = _tables(held, max(1, _cdiv(max(lens), STATE_BLOCK)), g)
        span = case["ratio"] * case["kv_block"]
        held = torch.div(s["seq_lens"] + span - 1, span, rounding_mode="floor")
        s["kv_table"], _ = _tables(held, max(1, _cdiv(max(lens), span)), g)
        s["maps"] = {
            "query_start": torch.empty(n + 1, dtype=torch.int32, device="cuda"),
            "token_to_req_indices": torch.empty(tokens, dtype=torch.int32, device="cuda"),
            "positions": torch.empty(tokens, dtype=torch.int64, device="cuda"),
            "slot_mapping": torch.empty(tokens, dtype=torch.int64, device="cuda"),
            "kv_slot_mapping": torch.empty(tokens, dtype=torch.int64, device="cuda"),
            "kv_lens": torch.empty(n, dtype=torch.int32, device="cuda"),
        }
    elif op == "decode":
        lens, block, heads = _lengths(n, case["longest"], case["spread"]), case["kv_block"], case["heads"]
        s["kv_lens"] = _ints(lens, order)
        held = torch.div(s["kv_lens"] + block - 1, block, rounding_mode="floor")
        s["block_table"], _ = _tables(held, max(1, _cdiv(max(lens), block)), g, spare=2)
        s["k_cache"] = _cache((int(held.sum()) + 2) * block, block, g)
        s["q"] = (2 * torch.randn(n, heads, HEAD, generator=g, device="cuda")).to(torch.bfloat16)
        s["sink"] = torch.randn(heads, generator=g, device="cuda") if case["sink"] else None
        s["scale"] = HEAD ** -0.5
        s["out"] = torch.empty(n, heads, HEAD, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(n, heads, dtype=torch.float32, device="cuda")
    else:
        shape = (case["parts"], n, case["heads"])
        s["part_out"] = torch.randn(*shape, HEAD, generator=g, device="cuda").to(torch.bfloat16)
        s["part_lse"] = 3 * torch.randn(*shape, generator=g, device="cuda")
        # a part that saw nothing: zeros, and a log-sum-exp of minus infinity
        nothing = torch.rand(*shape, generator=g, device="cuda") < 0.1
        s["part_out"][nothing] = 0
        s["part_lse"][nothing] = -math.inf
        s["out"] = torch.empty(n, case["heads"], HEAD, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(n, case["heads"], dtype=torch.float32, device="cuda") if case["lse"] else None
    if own:  # the handle that a serving loop keeps: argument descriptors (and the workspace of `decode`), no data
        s["call"] = _handle(s)
    return s


def _handle(s):
    from deepseek_v4_sparse_c128_gb300 import binding
    case = s["case"]
    if s["op"] == "tables":
        return binding.PreparedOp("extend_block_tables", s["seq_lens"], s["held"], s["block_table"], s["free_blocks"],
                                  s["taken"], case["ratio"], case["block"], held_out=s["held_out"],
                                  taken_out=s["taken_out"])
    if s["op"] == "maps":
        return binding.PreparedOp("build_slot_maps", s["seq_lens"], s["query_lens"], s["state_table"], STATE_BLOCK,
                                  s["kv_table"], case["kv_block"], case["ratio"], **s["maps"])
    if s["op"] == "decode":
        return binding.PreparedOp("decode_attention", s["q"], s["k_cache"], case["kv_block"], s["block_table"],
                                  s["kv_lens"], s["scale"], s["out"], lse=s["lse"], sink=s["sink"])
    return binding.PreparedOp("merge_attention", s["part_out"], s["part_lse"], s["out"], lse=s["lse"])


# ------------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["op"]
    if own:
        state["call"]()
        if op == "tables":
            return state["block_table"], state["held_out"], state["taken_out"]
        if op == "maps":
            return state["maps"]
        return (state["out"], state["lse"]) if state["lse"] is not None else (state["out"],)
    return {"tables": _plain_tables, "maps": _plain_maps, "decode": _plain_decode, "merge": _plain_merge}[op](state)


def _plain_tables(s):
    case, table, held = s["case"], s["block_table"], s["held"].long()
    entries = torch.div(s["seq_lens"].long(), case["ratio"], rounding_mode="floor")
    need = (torch.div(entries + case["block"] - 1, case["block"], rounding_mode="floor") - held).clamp_min(0)
    end = need.cumsum(0)
    need = torch.where(end <= s["free_blocks"].numel() - s["taken"], need, 0)
    column = torch.arange(table.shape[1], device="cuda")[None, :] - held[:, None]
    new = (column >= 0) & (column < need[:, None])
    at = (s["taken"] + (end - need)[:, None] + column).clamp(0, s["free_blocks"].numel() - 1)
    table.copy_(torch.where(new, s["free_blocks"][at], table))
    return table, (held + need).to(torch.int32), s["taken"] + need.sum()


def _slots(table, request, index, block, wanted):
    """table[request, index // block] * block + index % block where wanted, else -1."""
    column = torch.div(index, block, rounding_mode="floor").clamp(0, table.shape[1] - 1)
    return torch.where(wanted, table[request, column].long() * block + index % block, -1)


def _plain_maps(s):
    case, tokens = s["case"], s["maps"]["positions"].numel()
    end = s["query_lens"].long().cumsum(0)
    t = torch.arange(tokens, device="cuda")
    real = t < end[-1]
    request = torch.where(real, torch.searchsorted(end, t, right=True), 0)
    position = torch.where(real, s["seq_lens"].long()[request] - end[request] + t, 0)
    closes = real & ((position + 1) % case["ratio"] == 0)
    entry = torch.div(position, case["ratio"], rounding_mode="floor")
    return {
        "query_start": torch.cat([end.new_zeros(1), end]).to(torch.int32),
        "token_to_req_indices": request.to(torch.int32),
        "positions": position,
        "slot_mapping": _slots(s["state_table"], request, position, STATE_BLOCK, real),
        "kv_slot_mapping": _slots(s["kv_table"], request, entry, case["kv_block"], closes),
        "kv_lens": torch.div(s["seq_lens"], case["ratio"], rounding_mode="floor").to(torch.int32),
    }


def _plain_decode(s):
    cache, lens, block = s["k_cache"], s["kv_lens"].long(), s["case"]["kv_block"]
    index = torch.arange(s["block_table"].shape[1] * block, device="cuda")
    real = index[None, :] < lens[:, None]
    page = s["block_table"][:, torch.div(index, block, rounding_mode="floor")].long().clamp_min(0)
    stride = block * (RECORD + SCALES)
    data = cache.as_strided((cache.shape[0], block, RECORD), (stride, RECORD, 1))[page, index % block]
    power = cache.as_strided((cache.shape[0], block, SCALES), (stride, SCALES, 1), block * RECORD)[page, index % block]
    # 2^(byte - 127) is the float whose exponent field is the byte
    power = (power[..., : NOPE // GROUP].int() << 23).view(torch.float32)
    nope = data[..., :NOPE].contiguous().view(torch.float8_e4m3fn).float()
    nope = nope.unflatten(-1, (NOPE // GROUP, GROUP)) * power[..., None]
    k = torch.cat([nope.flatten(-2), data[..., NOPE:].contiguous().view(torch.bfloat16).float()], -1)
    k = torch.where(real[..., None], k, 0.0)
    score = torch.matmul(s["q"].float(), k.transpose(1, 2)) * s["scale"]
    score = torch.where(real[:, None, :], score, -math.inf)
    top = score.amax(-1)
    if s["sink"] is not None:
        top = torch.maximum(top, s["sink"][None, :])
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top[..., None])
    total = p.sum(-1)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"][None, :] - top)
    out = torch.matmul(p, k) / torch.where(total > 0, total, 1.0)[..., None]
    return out.to(torch.bfloat16), top + torch.log(total)


def _plain_merge(s):
    lse, part = s["part_lse"], s["part_out"].float()
    top = lse.amax(0)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = torch.exp(lse - top)
    total = weight.sum(0)
    part = torch.where((weight > 0)[..., None], part, 0.0)
    out = (part * weight[..., None]).sum(0) / torch.where(total > 0, total, 1.0)[..., None]
    out = out.to(torch.bfloat16)
    return (out, top + torch.log(total)) if s["lse"] is not None else (out,)


# ------------------------------------------------------------------------------------------ in 64 bits
def _e4m3_values():
    """The value of each e4m3 byte, from the format: sign, 4 exponent bits of bias 7, 3 mantissa bits, 0x7f NaN."""
    def value(b):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if b & 127 == 127 else math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        return -v if b & 128 else v
    return torch.tensor([value(b) for b in range(256)], dtype=torch.float64, device="cuda")


def _exact_decode(s):
    values, block, cache = _e4m3_values(), s["case"]["kv_block"], s["k_cache"]
    flat = cache.reshape(cache.shape[0], -1)
    outs, lses = [], []
    for r, n in enumerate(s["kv_lens"].tolist()):
        pages = flat[s["block_table"][r, : _cdiv(n, block)].long()]
        data = pages[:, : block * RECORD].reshape(-1, RECORD)[:n]
        scales = pages[:, block * RECORD:].reshape(-1, SCALES)[:n, : NOPE // GROUP]
        k = torch.empty(n, HEAD, dtype=torch.float64, device="cuda")
        k[:, :NOPE] = values[data[:, :NOPE].long()] * torch.pow(2.0, scales.double() - 127).repeat_interleave(GROUP, 1)
        k[:, NOPE:] = data[:, NOPE:].contiguous().view(torch.bfloat16).double()
        logits = s["q"][r].double() @ k.T * s["scale"]
        if s["sink"] is not None:  # one more logit with a value of zero
            logits = torch.cat([logits, s["sink"].double()[:, None]], 1)
            k = torch.cat([k, k.new_zeros(1, HEAD)])
        lse = torch.logsumexp(logits, 1)
        outs.append(torch.exp(logits - torch.where(torch.isinf(lse), 0.0, lse)[:, None]) @ k)
        lses.append(lse)
    return torch.stack(outs), torch.stack(lses)


def exact(case, seed):
    if case["op"] in ("tables", "maps"):  # whole numbers
        return None
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(s)
    lse = torch.logsumexp(s["part_lse"].double(), 0)
    share = torch.exp(s["part_lse"].double() - torch.where(torch.isinf(lse), 0.0, lse))
    out = torch.einsum("prh,prhd->rhd", share, s["part_out"].double())
    return (out, lse) if case["lse"] else (out,)
