"""Cases of the operators that carry a step's queries and keys past the recent tokens, for timing and comparison.

Three operators, each in a plain form (elementary torch operations) and as the calls of this package:

* ``norm``    queries normalised for each head and turned by their position, keys too, which go into the paged cache;
* ``rotary``  positions as rotations: ``table`` makes the cosines and sines, ``rotate`` turns part of each head;
* ``window``  attention of each token to the last tokens before it and a few first ones of its request.

A case fixes the sizes and how long the requests are (the set of lengths); the seed draws the values, the order of
the requests and the order of the physical blocks.
"""
import math

import torch

own = False

HEAD, NOPE, ROPE, GROUP = 512, 448, 64, 64   # head size, its FP8 part, its rotated part, columns per UE8M0 scale
RECORD, SCALES = 576, 8                      # bytes of an entry's data and of its scales
EPS = 1e-6
THETA = 10000.0
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one request's new token in a decode step: latency counts
        {"name": "norm_one", "op": "norm", "tokens": 1, "pad": 0, "heads": 64, "longest": 16374, "kv_block": 64,
         "weight": False, "dtype": "bf16"},
        # a decode step of 200 requests, padded to the size that the captured graph was made for
        {"name": "norm_batch", "op": "norm", "tokens": 200, "pad": 56, "heads": 128, "longest": 131072, "kv_block": 2,
         "weight": True, "dtype": "bf16"},
        # a chunk of prompts
        {"name": "norm_prefill", "op": "norm", "tokens": 7777, "pad": 0, "heads": 64, "longest": 16384, "kv_block": 64,
         "weight": False, "dtype": "bf16"},
        # the table of a model without scaling, 16 Ki positions
        {"name": "table_short", "op": "table", "positions": 16384, "begin": 0, "width": 64, "scaling": "none",
         "factor": 1.0},
        # the table of a million positions, stretched out of 64 Ki
        {"name": "table_long", "op": "table", "positions": 1048576, "begin": 0, "width": 64, "scaling": "yarn",
         "factor": 16.0},
        # a decode step's results, turned back (entries are values too, so results carry their positions)
        {"name": "rotate_batch", "op": "rotate", "tokens": 64, "heads": 64, "width": 512, "turned": 64, "first": 448,
         "layout": "pairs", "inverse": True, "longest": 131072, "dtype": "bf16"},
        # a prefill's results, turned back
        {"name": "rotate_prefill", "op": "rotate", "tokens": 4096, "heads": 64, "width": 512, "turned": 64, "first": 448,
         "layout": "pairs", "inverse": True, "longest": 16384, "dtype": "bf16"},
        # queries of a head of 128 whose first half turns, in the layout of halves, an odd number of tokens
        {"name": "rotate_halves", "op": "rotate", "tokens": 4099, "heads": 40, "width": 128, "turned": 64, "first": 0,
         "layout": "halves", "inverse": False, "longest": 65536, "dtype": "fp32"},
        # one request's new token: latency counts
        {"name": "window_one", "op": "window", "requests": 1, "longest": 16374, "spread": "full", "query": 1, "pad": 0,
         "heads": 64, "window": 128, "first": 0, "kv_block": 64, "sink": False},
        # a decode step of 200 requests, some of them shorter than the window, padded to a captured size
        {"name": "window_batch", "op": "window", "requests": 200, "longest": 8192, "spread": "skew", "query": 1,
         "pad": 56, "heads": 64, "window": 128, "first": 4, "kv_block": 64, "sink": True},
        # prompts and parts of prompts, about 5 thousand new tokens
        {"name": "window_prefill", "op": "window", "requests": 5, "longest": 2048, "spread": "even", "query": 2048,
         "pad": 0, "heads": 64, "window": 128, "first": 4, "kv_block": 64, "sink": True},
        # a few tokens at once (drafts to verify), few heads on this GPU, a window far longer than a tile
        {"name": "window_long", "op": "window", "requests": 16, "longest": 32768, "spread": "even", "query": 4, "pad": 0,
         "heads": 16, "window": 4096, "first": 4, "kv_block": 16, "sink": False},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "table", "rotate", "rotate", "window", "window", "window"])
    if op == "norm":
        tokens = _log_uniform(rng, 1, 8192)
        return {"op": op, "tokens": tokens, "pad": rng.choice([0, rng.randint(1, 60)]),
                "heads": _log_uniform(rng, 1, max(1, min(128, 248000 // tokens))), "longest": _log_uniform(rng, 1, 1 << 17),
                "kv_block": rng.choice([1, 2, 16, 64, 67]), "weight": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "table":
        scaling = rng.choice(["none", "linear", "yarn"])
        width = rng.choice([32, 64, 96, 128])
        return {"op": op, "positions": _log_uniform(rng, 1, (1 << 26) // width), "begin": rng.choice([0, rng.randint(1, 1 << 20)]),
                "width": width, "scaling": scaling, "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 40.0])}
    if op == "rotate":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        width = rng.choice([64, 96, 128, 192, 512])
        turned = rng.choice([t for t in (32, 64, 96, 128) if t <= width])
        tokens = _log_uniform(rng, 1, 8192)
        most = (1 << 27) // (width * tokens * (2 if dtype == "fp32" else 1))
        return {"op": op, "tokens": tokens, "heads": _log_uniform(rng, 1, max(1, min(128, most))), "width": width, "turned": turned,
                "first": rng.choice([0, width - turned, (width - turned) // 2]), "layout": rng.choice(["pairs", "halves"]),
                "inverse": rng.random() < 0.5, "longest": _log_uniform(rng, 1, 1 << 17), "dtype": dtype}
    window = rng.choice([128, 128, _log_uniform(rng, 1, 4096)])
    first = rng.choice([0, 0, 4, rng.randint(1, 16)])
    heads, query = _log_uniform(rng, 1, 128), rng.choice([1, 1, rng.randint(2, 8), _log_uniform(rng, 2, 2048)])
    # the rows (a token's head each) times the entries that they see, and the tokens times those, are bounded
    most = max(1, min(4400, 34000000 // (heads * (window + first)), 580000 // (window + first)))
    query = min(query, most)
    requests = max(1, min(256, most // query))
    requests = _log_uniform(rng, max(1, requests // 4), requests)
    return {"op": op, "requests": requests, "longest": max(query, _log_uniform(rng, 1, 1 << 15)),
            "spread": rng.choice(["full", "even", "skew"]), "query": query, "pad": rng.choice([0, rng.randint(1, 60)]),
            "heads": heads, "window": window, "first": first, "kv_block": rng.choice([1, 2, 16, 64, 67]),
            "sink": rng.random() < 0.5}


def _lengths(n, longest, spread):
    """The n lengths of a case, 0 .. longest: all the longest, evenly spread, or most of them short."""
    if spread == "full":
        return [longest] * n
    if spread == "even":
        return [max(1, longest * (i + 1) // n) for i in range(n)]
    return [int(longest * (i / n) ** 3) for i in range(n - 1)] + [longest]


def _queries(case):
    """New tokens of each request: the same few of all, or 0 .. query (the longest request has `query`)."""
    lens, query = _lengths(case["requests"], case["longest"], case["spread"]), case["query"]
    if query <= 8:
        return [min(query, n) for n in lens]
    return [min(n, query * ((7 * i) % 11) // 10) for i, n in enumerate(lens[:-1])] + [query]


def _cdiv(a, b):
    return -(-a // b)


def _seen(p, case):
    """Entries that the token at position p sees."""
    return min(p + 1, case["window"]) + min(case["first"], max(0, p + 1 - case["window"]))


def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": 4 * case["positions"] * case["width"], "flops": 8 * case["positions"] * case["width"]}
    if op == "rotate":
        values = case["tokens"] * case["heads"] * case["width"]
        return {"bytes": 2 * values * (4 if case["dtype"] == "fp32" else 2) + case["tokens"] * (8 + 4 * case["turned"]),
                "flops": 3 * case["tokens"] * case["heads"] * case["turned"]}
    if op == "norm":
        item, rows = 4 if case["dtype"] == "fp32" else 2, case["tokens"] * case["heads"]
        return {"bytes": rows * HEAD * (item + 2) + case["tokens"] * (HEAD * item + RECORD + SCALES + 16 + 4 * ROPE)
                + 4 * HEAD * (1 + case["weight"]),
                "flops": (rows + case["tokens"]) * HEAD * (4 if case["weight"] else 3)}
    lens, new = _lengths(case["requests"], case["longest"], case["spread"]), _queries(case)
    tokens = sum(new)
    # a request's entries that any of its tokens sees
    entries = 0
    for n, q in zip(lens, new):
        if q:
            begin = max(0, n - q - case["window"] + 1)
            entries += n - begin + min(case["first"], begin)
    pairs = sum(_seen(p, case) for n, q in zip(lens, new) for p in range(n - q, n))
    return {"bytes": entries * (RECORD + SCALES) + 4 * _cdiv(entries, case["kv_block"]) + tokens * 20
            + tokens * case["heads"] * (4 * HEAD + 4) + (4 * case["heads"] if case["sink"] else 0),
            "flops": 4 * HEAD * case["heads"] * pairs}


# ------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _angles_table(rows, width):
    """Cosines and sines [rows, width] of positions 0 .. rows - 1, as a model keeps them."""
    step = THETA ** (-torch.arange(0, width, 2, dtype=torch.float64, device="cuda") / width)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * step
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _cache(entries, block, g):
    """A cache of `entries` records (whole blocks): FP8 e4m3 in groups of 64 with UE8M0 scales, the last 64 columns
    bf16. Vectors as they come out of an RMSNorm with a weight near one."""
    x = _randn(g, entries, HEAD) * (1 + 0.1 * _randn(g, HEAD))
    nope = x[:, :NOPE].reshape(entries, NOPE // GROUP, GROUP)
    e = torch.ceil(torch.log2(nope.abs().amax(-1).clamp_min(1e-4) / 448))
    codes = (nope * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(entries, NOPE)
    rope = x[:, NOPE:].to(torch.bfloat16).view(torch.uint8)
    data = torch.cat([codes, rope], 1).reshape(entries // block, block * RECORD)
    scales = torch.zeros(entries, SCALES, dtype=torch.uint8, device="cuda")
    scales[:, : NOPE // GROUP] = (e + 127).to(torch.uint8)
    cache = torch.cat([data, scales.reshape(entries // block, block * SCALES)], 1)
    return cache.reshape(entries // block, block, RECORD + SCALES)


def _records(cache):
    """A cache's records and scales as byte views [blocks, block, 576] and [blocks, block, 8]."""
    n, block = cache.shape[:2]
    stride = block * (RECORD + SCALES)
    return (cache.as_strided((n, block, RECORD), (stride, RECORD, 1)),
            cache.as_strided((n, block, SCALES), (stride, SCALES, 1), block * RECORD))


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"op": op, "case": case}
    if op == "table":
        s["begin"] = case["begin"] + seed % 97
        s["rope"] = {"theta": THETA * (1 + 0.01 * (seed % 97)), "scaling": case["scaling"], "factor": case["factor"],
                     "original_positions": 65536, "beta_fast": 32.0, "beta_slow": 1.0,
                     "magnitude": 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0}
        s["table"] = torch.empty(case["positions"], case["width"], device="cuda")
    elif op == "rotate":
        s["x"] = _randn(g, case["tokens"], case["heads"], case["width"]).to(TYPES[case["dtype"]])
        s["positions"] = torch.randint(case["longest"], (case["tokens"],), generator=g, device="cuda")
        s["cos_sin"] = _angles_table(case["longest"], case["turned"])
        s["out"] = torch.empty_like(s["x"])
    elif op == "norm":
        tokens, pad, block, kind = case["tokens"], case["pad"], case["kv_block"], TYPES[case["dtype"]]
        n = tokens + pad
        # projections: each head at a scale of its own
        s["q"] = (_randn(g, n, case["heads"], HEAD) * torch.exp(0.3 * _randn(g, case["heads"], 1))).to(kind)
        s["k"] = (3 * _randn(g, n, HEAD)).to(kind)
        s["q_weight"] = 1 + 0.1 * _randn(g, HEAD) if case["weight"] else None
        s["k_weight"] = 1 + 0.1 * _randn(g, HEAD)
        s["positions"] = torch.randint(case["longest"], (n,), generator=g, device="cuda")
        s["cos_sin"] = _angles_table(case["longest"], ROPE)
        blocks = _cdiv(tokens, block) + 1
        s["k_cache"] = torch.zeros(blocks, block, RECORD + SCALES, dtype=torch.uint8, device="cuda")
        s["slots"] = torch.randperm(blocks * block, generator=g, device="cuda")[:n]
        if pad:  # rows behind the last token
            s["slots"] = torch.cat([s["slots"][:tokens], s["slots"].new_full((pad,), -1)])
            s["positions"][tokens:] = 0
        s["q_out"] = torch.zeros(n, case["heads"], HEAD, dtype=torch.bfloat16, device="cuda")
        # the cache by what its bytes stand for
        data, scales = _records(s["k_cache"])
        s["stored"] = {"codes": data[..., :NOPE].view(torch.float8_e4m3fn), "rope": data[..., NOPE:].view(torch.bfloat16),
                       "scales": scales[..., : NOPE // GROUP].view(torch.float8_e8m0fnu)}
    else:
        n, block = case["requests"], case["kv_block"]
        order = torch.randperm(n, generator=g, device="cuda")
        lens = torch.tensor(_lengths(n, case["longest"], case["spread"]), device="cuda")[order]
        new = torch.tensor(_queries(case), device="cuda")[order]
        tokens = sum(_queries(case))
        request = torch.repeat_interleave(torch.arange(n, device="cuda"), new, output_size=tokens)
        position = torch.arange(tokens, device="cuda") - (new.cumsum(0) - lens)[request]
        # blocks that no token of this step sees are not held any more
        begin = (lens - new - case["window"] + 1).clamp_min(0)
        at = torch.arange(max(1, _cdiv(case["longest"], block)), device="cuda") * block
        held = (at < lens[:, None]) & ((at + block > begin[:, None]) | (at < case["first"]))
        total = int(held.sum())
        s["block_table"] = torch.full(held.shape, -1, dtype=torch.int32, device="cuda")
        s["block_table"][held] = torch.randperm(total + 2, generator=g, device="cuda").to(torch.int32)[:total]
        s["k_cache"] = _cache((total + 2) * block, block, g)
        pad = case["pad"]
        s["requests"] = torch.cat([request, request.new_zeros(pad)]).to(torch.int32)
        s["positions"] = torch.cat([position, position.new_zeros(pad)])
        slot = s["block_table"][request, torch.div(position, block, rounding_mode="floor")].long() * block + position % block
        s["slots"] = torch.cat([slot, slot.new_full((pad,), -1)])
        s["q"] = (2 * _randn(g, tokens + pad, case["heads"], HEAD)).to(torch.bfloat16)
        s["sink"] = _randn(g, case["heads"]) if case["sink"] else None
        s["scale"] = HEAD ** -0.5
        s["out"] = torch.zeros(tokens + pad, case["heads"], HEAD, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(tokens + pad, case["heads"], device="cuda")
    if own:  # the handle that a serving loop keeps: argument descriptors (and the workspace of `window`), no data
        s["call"] = _handle(s)
    return s


def _handle(s):
    from deepseek_v4_sparse_c128_gb300 import binding
    case = s["case"]
    if s["op"] == "table":
        return binding.PreparedOp("build_cos_sin", binding.rope(**s["rope"]), s["begin"], s["table"])
    if s["op"] == "rotate":
        return binding.PreparedOp("rotate", s["x"], s["positions"], s["cos_sin"], s["out"], first_column=case["first"],
                                  layout=binding.ROPE_PAIRS if case["layout"] == "pairs" else binding.ROPE_HALVES,
                                  inverse=case["inverse"])
    if s["op"] == "norm":
        return binding.PreparedOp("norm_rope_store", s["positions"], s["slots"], EPS, s["cos_sin"], q=s["q"], q_w=s["q_weight"],
                                  q_out=s["q_out"], k=s["k"], k_w=s["k_weight"], k_cache=s["k_cache"],
                                  kv_block_size=case["kv_block"])
    return binding.PreparedOp("window_attention", s["q"], s["k_cache"], case["kv_block"], s["block_table"], s["requests"],
                              s["positions"], s["slots"], case["window"], s["scale"], s["out"], first=case["first"],
                              lse=s["lse"], sink=s["sink"])


# ------------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["op"]
    if own:
        state["call"]()
        if op == "table":
            return state["table"]
        if op == "rotate":
            return state["out"]
        if op == "norm":
            return {"q": state["q_out"], **state["stored"]}
        return state["out"], state["lse"]
    return {"table": _plain_table, "rotate": _plain_rotate, "norm": _plain_norm, "window": _plain_window}[op](state)


def _steps(rope, width):
    """Radians per position of each pair (64 bits). yarn: pairs that turn more than beta_fast times over the original
    positions keep their step, those under beta_slow turns are stretched by the factor, with a ramp between."""
    pair = torch.arange(width // 2, dtype=torch.float64, device="cuda")
    step = torch.exp(pair * (-2 * math.log(rope["theta"]) / width))
    if rope["scaling"] == "linear":
        return step / rope["factor"]
    if rope["scaling"] == "yarn":
        def pair_of(turns):
            return width * math.log(rope["original_positions"] / (2 * math.pi * turns)) / (2 * math.log(rope["theta"]))
        low = max(math.floor(pair_of(rope["beta_fast"])), 0)
        high = min(math.ceil(pair_of(rope["beta_slow"])), width - 1)
        ramp = ((pair - low) / max(high - low, 0.001)).clamp(0, 1)
        return step * (1 - ramp) + step / rope["factor"] * ramp
    return step


def _plain_table(s):
    rope, case = s["rope"], s["case"]
    position = torch.arange(s["begin"], s["begin"] + case["positions"], dtype=torch.float64, device="cuda")
    angle = position[:, None] * _steps(rope, case["width"])
    return (torch.cat([angle.cos(), angle.sin()], 1) * rope["magnitude"]).float()


def _plain_rotate(s):
    case, x = s["case"], s["x"].float()
    cos, sin = s["cos_sin"][s["positions"]][:, None, :].chunk(2, -1)
    if case["inverse"]:
        sin = -sin
    a, b = case["first"], case["first"] + case["turned"]
    part = x[..., a:b]
    if case["layout"] == "pairs":
        u, v = part[..., 0::2], part[..., 1::2]
        part = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    else:
        u, v = part.chunk(2, -1)
        part = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    return torch.cat([x[..., :a], part, x[..., b:]], -1).to(s["x"].dtype)


def _turned(x, cos, sin):
    """x with its last 64 columns, pairs of neighbours, turned."""
    u, v = x[..., NOPE::2], x[..., NOPE + 1::2]
    return torch.cat([x[..., :NOPE], torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)], -1)


def _plain_norm(s):
    real = slice(s["case"]["tokens"])
    cos, sin = s["cos_sin"][s["positions"]].chunk(2, -1)
    q = s["q"].float()
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS)
    if s["q_weight"] is not None:
        q = q * s["q_weight"]
    q = _turned(q, cos[:, None, :], sin[:, None, :]).to(torch.bfloat16)
    q = torch.where((s["slots"] >= 0)[:, None, None], q, s["q_out"])
    # the mean square in 64 bits: the codes behind it are next to borders
    k = s["k"][real].float()
    var = k.double().square().mean(-1, keepdim=True).float()
    k = k * torch.rsqrt((var + EPS).double()).float() * s["k_weight"]
    k = _turned(k, cos[real], sin[real]).to(torch.bfloat16)
    nope = k[:, :NOPE].float().unflatten(-1, (NOPE // GROUP, GROUP))
    bits = (nope.abs().amax(-1).clamp_min(1e-4) * (1 / 448)).view(torch.int32)
    e = (bits >> 23) - 127 + ((bits & 0x7fffff) != 0).int()   # ceil(log2)
    codes = torch.ldexp(nope, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    block, cache = s["case"]["kv_block"], s["k_cache"]
    page, at = torch.div(s["slots"][real], block, rounding_mode="floor"), s["slots"][real] % block
    data, scales = _records(cache)
    data[page, at] = torch.cat([codes.flatten(-2).view(torch.uint8), k[:, NOPE:].contiguous().view(torch.uint8)], -1)
    scales[page, at] = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, 1))
    return {"q": q, **s["stored"]}


def _plain_window(s):
    case, block = s["case"], s["case"]["kv_block"]
    first, position = case["first"], s["positions"][:, None]
    begin = (position - case["window"] + 1).clamp_min(0)
    # the first entries that the window does not hold, then the window's
    at = torch.cat([torch.arange(first, device="cuda").expand(len(position), first),
                    begin + torch.arange(case["window"], device="cuda")], 1)
    seen = torch.cat([at[:, :first] < begin, at[:, first:] <= position], 1)
    column = torch.div(torch.where(seen, at, 0), block, rounding_mode="floor")
    page = s["block_table"][s["requests"].long()[:, None], column].long().clamp_min(0)
    data, power = (v[page, at % block] for v in _records(s["k_cache"]))
    # 2^(byte - 127) is the float whose exponent field is the byte
    power = (power[..., : NOPE // GROUP].int() << 23).view(torch.float32)
    nope = data[..., :NOPE].contiguous().view(torch.float8_e4m3fn).float()
    nope = nope.unflatten(-1, (NOPE // GROUP, GROUP)) * power[..., None]
    k = torch.cat([nope.flatten(-2), data[..., NOPE:].contiguous().view(torch.bfloat16).float()], -1)
    k = torch.where(seen[..., None], k, 0.0)
    score = torch.matmul(s["q"].float(), k.transpose(1, 2)) * s["scale"]
    score = torch.where(seen[:, None, :], score, -math.inf)
    top = score.amax(-1)
    if s["sink"] is not None:
        top = torch.maximum(top, s["sink"][None, :])
    p = torch.exp(score - top[..., None])
    total = p.sum(-1)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"][None, :] - top)
    out = torch.matmul(p, k) / total[..., None]
    real = (s["slots"] >= 0)[:, None]
    return (torch.where(real[..., None], out.to(torch.bfloat16), s["out"]), torch.where(real, top + torch.log(total), s["lse"]))


# ------------------------------------------------------------------------------------------ in 64 bits
def _e4m3_values():
    """The value of each e4m3 byte, from the format: sign, 4 exponent bits of bias 7, 3 mantissa bits, 0x7f NaN."""
    def value(b):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if b & 127 == 127 else math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        return -v if b & 128 else v
    return torch.tensor([value(b) for b in range(256)], dtype=torch.float64, device="cuda")


def _exact_window(s):
    case, block, first = s["case"], s["case"]["kv_block"], s["case"]["first"]
    values, flat = _e4m3_values(), s["k_cache"].flatten(1)
    out, lse = s["out"].double(), s["lse"].double()
    table = s["block_table"].long()
    for t, (r, p, slot) in enumerate(zip(s["requests"].tolist(), s["positions"].tolist(), s["slots"].tolist())):
        if slot < 0:
            continue
        begin = max(0, p + 1 - case["window"])
        at = torch.tensor([*range(min(first, begin)), *range(begin, p + 1)], device="cuda")
        page, within = table[r, torch.div(at, block, rounding_mode="floor")], at % block
        data = flat[page[:, None], within[:, None] * RECORD + torch.arange(RECORD, device="cuda")]
        power = flat[page[:, None], block * RECORD + within[:, None] * SCALES + torch.arange(NOPE // GROUP, device="cuda")]
        k = torch.empty(len(at), HEAD, dtype=torch.float64, device="cuda")
        k[:, :NOPE] = values[data[:, :NOPE].long()] * torch.pow(2.0, power.double() - 127).repeat_interleave(GROUP, 1)
        k[:, NOPE:] = data[:, NOPE:].contiguous().view(torch.bfloat16).double()
        logits = s["q"][t].double() @ k.T * s["scale"]
        if s["sink"] is not None:  # one more logit with a value of zero
            logits = torch.cat([logits, s["sink"].double()[:, None]], 1)
            k = torch.cat([k, k.new_zeros(1, HEAD)])
        lse[t] = torch.logsumexp(logits, 1)
        out[t] = torch.exp(logits - lse[t][:, None]) @ k
    return out, lse


def _turn(pairs, cos_sin):
    """Complex numbers times those of the angles."""
    half = cos_sin.shape[-1] // 2
    return pairs * torch.complex(cos_sin[..., :half].double(), cos_sin[..., half:].double())


def _exact_rotate(s):
    case, out = s["case"], s["x"].double()
    part = out[..., case["first"] : case["first"] + case["turned"]]
    cos_sin = s["cos_sin"].index_select(0, s["positions"])[:, None, :]
    if case["layout"] == "halves":
        part = part.unflatten(-1, (2, -1)).transpose(-1, -2)
    else:
        part = part.unflatten(-1, (-1, 2))
    z = torch.view_as_complex(part.contiguous())
    z = torch.view_as_real(_turn(z.conj(), cos_sin).conj().resolve_conj() if case["inverse"] else _turn(z, cos_sin))
    z = z.transpose(-1, -2) if case["layout"] == "halves" else z
    out[..., case["first"] : case["first"] + case["turned"]] = z.flatten(-2)
    return out


def _exact_norm(s):
    slots = s["slots"].tolist()

    def unit(x, weight):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / HEAD + EPS).sqrt()
        x = x * weight.double() if weight is not None else x
        turn = s["cos_sin"][s["positions"]]
        turn = turn[:, None, :] if x.dim() == 3 else turn
        z = torch.view_as_complex(x[..., NOPE:].unflatten(-1, (-1, 2)).contiguous())
        x[..., NOPE:] = torch.view_as_real(_turn(z, turn)).flatten(-2)
        return x

    q, k = unit(s["q"], s["q_weight"]), unit(s["k"], s["k_weight"])
    q[s["slots"] < 0] = 0
    # what the formats make of the vectors: each group of 64 by its scale to the nearest e4m3, the rest to bf16
    data, scales = _records(s["k_cache"])
    codes, rope = (torch.zeros(*data.shape[:2], w, dtype=torch.float64, device="cuda") for w in (NOPE, ROPE))
    power = torch.full((*data.shape[:2], NOPE // GROUP), 2.0 ** -127, dtype=torch.float64, device="cuda")
    group = k[:, :NOPE].bfloat16().double().unflatten(-1, (-1, GROUP))
    power2 = torch.exp2(torch.ceil(torch.log2(group.abs().amax(-1).clamp_min(1e-4) / 448)))
    near = _nearest_e4m3(group / power2[..., None]).flatten(1)
    block = s["case"]["kv_block"]
    live = [t for t, slot in enumerate(slots) if slot >= 0]
    at = torch.tensor([slots[t] for t in live], device="cuda")
    live = torch.tensor(live, device="cuda")
    where = (torch.div(at, block, rounding_mode="floor"), at % block)
    codes[where], rope[where], power[where] = near[live], k[live][:, NOPE:], power2[live]
    return {"q": q, "codes": codes, "rope": rope, "scales": power}


def _nearest_e4m3(x):
    values = torch.sort(_e4m3_values()[:127]).values  # 0 .. 448, by their byte
    index = torch.searchsorted(values, x.abs().contiguous()).clamp(1, 126)
    low, high = values[index - 1], values[index]
    up = (x.abs() - low > high - x.abs()) | ((x.abs() - low == high - x.abs()) & (index % 2 == 0))  # ties to the even byte
    return torch.where(up, high, low).copysign(x)


def _exact_table(s):
    rope, case, half = s["rope"], s["case"], s["case"]["width"] // 2
    steps = []
    for i in range(half):
        step = rope["theta"] ** (-2 * i / case["width"])
        if case["scaling"] != "none":
            keep = 0.0
            if case["scaling"] == "yarn":
                at = [case["width"] * math.log(rope["original_positions"] / (b * 2 * math.pi)) / (2 * math.log(rope["theta"]))
                      for b in (rope["beta_fast"], rope["beta_slow"])]
                low, high = max(0, math.floor(at[0])), min(case["width"] - 1, math.ceil(at[1]))
                keep = 1 - min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            step = step * keep + step / rope["factor"] * (1 - keep)
        steps.append(step)
    position = s["begin"] + torch.arange(case["positions"], device="cuda")
    angle = torch.outer(position.double(), torch.tensor(steps, dtype=torch.float64, device="cuda"))
    z = torch.polar(torch.full_like(angle, rope["magnitude"]), angle)
    return torch.cat([z.real, z.imag], 1)


def exact(case, seed):
    s = prepare(case, seed)
    return {"table": _exact_table, "rotate": _exact_rotate, "norm": _exact_norm, "window": _exact_window}[case["op"]](s)
