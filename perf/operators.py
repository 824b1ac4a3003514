"""The serving operators between the q/k/v projections and the output projection, as cases that can be timed.

Four operators of one decode or prefill step over a paged key-value cache:

* ``slots``    block tables and slot maps from request lengths;
* ``append``   per-head norms of q and k, position rotation, and the write of k and v into the cache;
* ``decode``   attention of one new token a request over its pages;
* ``prefill``  causal attention of a chunk of new tokens over the same pages.

The cache is ``[pages, heads, page_size, dim]`` in bf16, or int8 codes of that shape with one fp32 scale for every 32
values of a head.  With ``own`` false, ``run`` is elementary torch in fp32; with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

BLOCK = 32


# ---- the cases -----------------------------------------------------------------------------------------------------

def listed():
    return [
        # One user's decode step shortly after a prompt: 32 full heads of 128 (the 4096-wide projections).  Latency.
        {"name": "decode_one_user", "op": "decode", "requests": 1, "length": 203, "spread": 1.0, "heads": 32,
         "kv_heads": 32, "dim": 128, "page": 16, "cache": "bf16", "window": 0, "sinks": 0, "idle": 0, "layout": 1},
        # A decode batch of the library's 16 rows, shared heads, quantized cache, ragged lengths.
        {"name": "decode_batch_q8", "op": "decode", "requests": 16, "length": 8191, "spread": 0.25, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "cache": "q8", "window": 0, "sinks": 0, "idle": 1, "layout": 2},
        # Streaming chats whose context outgrew a sliding window; the first four tokens stay visible.  Narrow heads,
        # pages that end inside a tile.
        {"name": "decode_window", "op": "decode", "requests": 64, "length": 30001, "spread": 0.1, "heads": 24,
         "kv_heads": 8, "dim": 64, "page": 48, "cache": "bf16", "window": 4096, "sinks": 4, "idle": 0, "layout": 3},
        # One long document: all the work is along the cache.
        {"name": "decode_long", "op": "decode", "requests": 1, "length": 131072, "spread": 1.0, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 128, "cache": "bf16", "window": 0, "sinks": 0, "idle": 0, "layout": 4},
        # One 512-row prefill chunk (the largest the projections take) after 4096 cached tokens, full heads.
        {"name": "prefill_chunk", "op": "prefill", "requests": 1, "rows": 512, "length": 4096, "spread": 1.0,
         "heads": 32, "kv_heads": 32, "dim": 128, "page": 16, "cache": "bf16", "window": 0, "sinks": 0, "layout": 5},
        # Several requests' rows in one chunk over a quantized cache, odd counts.
        {"name": "prefill_ragged_q8", "op": "prefill", "requests": 5, "rows": 509, "length": 6007, "spread": 0.3,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 32, "cache": "q8", "window": 0, "sinks": 0, "layout": 6},
        # A prompt through a layer with a sliding window and sinks, narrow heads.
        {"name": "prefill_window", "op": "prefill", "requests": 2, "rows": 4097, "length": 2000, "spread": 0.5,
         "heads": 24, "kv_heads": 8, "dim": 64, "page": 48, "cache": "bf16", "window": 1024, "sinks": 4, "layout": 7},
        # A whole prompt in one call, causal: the largest product.
        {"name": "prefill_prompt", "op": "prefill", "requests": 1, "rows": 8192, "length": 0, "spread": 1.0,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cache": "bf16", "window": 0, "sinks": 0, "layout": 8},
        # The append of a 16-row decode step: 32 full heads, halves rotated, no norms.
        {"name": "append_decode", "op": "append", "rows": 16, "heads": 32, "kv_heads": 32, "dim": 128, "page": 16,
         "rotary": 128, "interleaved": False, "norm": False, "positions": 8192, "layout": 9},
        # The append of a long prompt: per-head norms, pairs rotated in part of the head, some rows padding.
        {"name": "append_prompt", "op": "append", "rows": 8191, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64,
         "rotary": 64, "interleaved": True, "norm": True, "positions": 131072, "layout": 10},
        # Slots of a 16-request decode step.
        {"name": "slots_decode", "op": "slots", "requests": 16, "rows": 16, "capacity": 16, "length": 8192,
         "page": 16, "layout": 11},
        # Slots of a mixed step of a large server: many decodes, some long prompts, padding rows at the end.
        {"name": "slots_mixed", "op": "slots", "requests": 1500, "rows": 30011, "capacity": 32768, "length": 20000,
         "page": 64, "layout": 12},
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))
    n = min(hi, max(lo, n))
    return n + 1 if n == 3072 else n


HEADS = [(32, 32), (32, 8), (24, 8), (16, 2), (8, 1), (28, 4), (40, 8), (12, 12), (32, 1)]


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "slots"])
    layout = rng.randrange(1 << 30)
    heads, kv_heads = rng.choice(HEADS)
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "slots":
        requests = _log_int(rng, 1, 2000)
        rows = _log_int(rng, max(1, requests // 2), 32000)
        return {"op": op, "requests": requests, "rows": rows, "capacity": rows + rng.choice([0, 0, 7, 500]),
                "length": _log_int(rng, 16, 20000), "page": page, "layout": layout}
    if op == "append":
        return {"op": op, "rows": _log_int(rng, 1, 8191), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "page": page, "rotary": rng.choice([dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.5,
                "norm": rng.random() < 0.5, "positions": _log_int(rng, 4096, 131072), "layout": layout}
    window = rng.choice([0, 0, _log_int(rng, 64, 4096)])
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "cache": rng.choice(["bf16", "q8"]), "window": window, "sinks": rng.choice([0, 4, 17]) if window else 0,
            "spread": rng.choice([1.0, 0.5, 0.1]), "layout": layout}
    if op == "decode":
        case["requests"] = _log_int(rng, 1, 64)
        # at most the cache of the longest listed context
        most = max(1, 131072 * 8 * 128 // (kv_heads * dim * case["requests"]))
        case["length"] = _log_int(rng, 1, min(131072, most))
        case["idle"] = 1 if case["requests"] >= 3 and rng.random() < 0.3 else 0
        return case
    case["requests"] = rng.choice([1, 1, 2, 5, 9])
    case["rows"] = _log_int(rng, case["requests"], 4099)
    # at most the pairs of the largest listed prompt, padding of the batch included
    most = 8192 * 8192 * 32 // (2 * heads * case["rows"] * case["requests"])
    case["length"] = _log_int(rng, 1, max(1, min(30000, most)))
    return case


def _split(rng, total, parts):
    """`total` rows over `parts` requests, each at least one while they last, unevenly."""
    if parts > total:
        return [1] * total + [0] * (parts - total)
    weights = [rng.uniform(0.3, 1.0) for _ in range(parts)]
    room = total - parts
    counts = [1 + int(room * w / sum(weights)) for w in weights]
    counts[0] += total - sum(counts)
    return counts


def _spread(rng, case, n):
    """n lengths up to case["length"], at least `spread` of it; the first one is the full length."""
    top = case["length"]
    low = max(1, int(top * case["spread"])) if top else 0
    return [top] + [rng.randint(low, top) if top else 0 for _ in range(n - 1)]


def _requests(case):
    """(cached, fresh) lengths of the case's requests, from the case alone."""
    rng = random.Random(case["layout"])
    n = case["requests"]
    if case["op"] == "decode":
        lens = _spread(rng, case, n)
        for i in range(case["idle"]):
            lens[1 + i] = 0  # a slot of the batch with no request in it
        return [max(0, x - 1) for x in lens], [1 if x else 0 for x in lens]
    if case["op"] == "prefill":
        return _spread(rng, case, n), _split(rng, case["rows"], n)
    fresh = _split(rng, case["rows"], n)
    return [rng.randint(0, case["length"]) for _ in range(n)], fresh


def _pages_of(n, page):
    return (n + page - 1) // page


# ---- what a program has in hand before the call --------------------------------------------------------------------

def _quantize(x):
    d = x.abs().amax(-1) / 127.0
    q = torch.where(d[..., None] > 0, torch.round(x / d[..., None]), torch.zeros_like(x))
    return q.clamp(-127, 127).to(torch.int8), d


def _cache_of(case, gen, pages):
    """Keys and values of all pages: keys with a few strong channels, as heads have; pages in shuffled use."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    out = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        if name == "k":
            gain = torch.ones(case["dim"], device="cuda")
            gain[:: case["dim"] // 4] = 3.0
            x *= gain
        if case["cache"] == "q8":
            q, d = _quantize(x.view(*shape[:-1], case["dim"] // BLOCK, BLOCK))
            out[name], out[name + "_scale"] = q.view(shape), d.contiguous()
        else:
            out[name] = x.to(torch.bfloat16)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + case["layout"] % 1000003)
    rng = random.Random(seed * 31 + case["layout"])
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    state = {"case": case, "op": case["op"]}
    if case["op"] == "append":
        rows, page, dim = case["rows"], case["page"], case["dim"]
        pages = 2 * _pages_of(rows, page) + 1
        for name, n in (("q", case["heads"]), ("k", case["kv_heads"]), ("v", case["kv_heads"])):
            state[name] = torch.randn((rows, n * dim), generator=gen, device="cuda") * 1.7
        for name in ("k", "v"):
            shape = (pages, case["kv_heads"], page, dim)
            state[name + "_cache"] = torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
        start = rng.randint(0, max(0, case["positions"] - rows))
        pos = torch.arange(start, start + rows, device="cuda", dtype=torch.int32) % case["positions"]
        slots = torch.randperm(pages * page, generator=gen, device="cuda")[:rows]
        idle = rows // 50  # rows of a fixed-size batch that hold no token
        if idle:
            pos[rows - idle:] = -1
            slots[rows - idle:] = -1
        state["positions"], state["slots"] = pos, slots
        half = case["rotary"] // 2
        freq = 500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        angle = torch.arange(case["positions"], dtype=torch.float64)[:, None] * freq
        state["table"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).cuda()
        for name in ("q_gamma", "k_gamma"):
            gamma = 0.5 + torch.rand(dim, generator=gen, device="cuda")
            state[name] = gamma if case["norm"] else None
        return state
    cached, fresh = _requests(case)
    page = case["page"]
    if case["op"] == "slots":
        have = [_pages_of(c, page) for c in cached]
        want = [_pages_of(c + f, page) for c, f in zip(cached, fresh)]
        total = sum(want) + 64
        order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
        used = sum(have)
        table = torch.full((len(cached), max(max(want), 1) + 3), -1, dtype=torch.int32, device="cuda")
        cols = torch.arange(table.shape[1], device="cuda")
        mask = cols[None, :] < ints(have)[:, None]
        table[mask] = order[:used]
        state.update(cached=ints(cached), fresh=ints(fresh), table=table, free=order[used:].contiguous(),
                     head=ints([rng.randint(0, 8)]))
        return state
    lens = [c + f for c, f in zip(cached, fresh)]
    counts = [_pages_of(n, page) for n in lens]
    width = max(max(counts), 1)
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    mask = torch.arange(width, device="cuda")[None, :] < ints(counts)[:, None]
    table[mask] = order[: sum(counts)]
    state.update(_cache_of(case, gen, pages))
    rows = len(lens) if case["op"] == "decode" else sum(fresh)
    q = torch.randn((rows, case["heads"] * case["dim"]), generator=gen, device="cuda") * 1.5
    starts = [0]
    for f in fresh:
        starts.append(starts[-1] + f)
    state.update(q=q.to(torch.bfloat16), table=table, lens=ints(lens), row_start=ints(starts), most=max(fresh),
                 scale=1.0 / math.sqrt(case["dim"]))
    return state


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"slots": _plain_slots, "append": _plain_append, "decode": _plain_decode,
            "prefill": _plain_prefill}[state["op"]](state)


def _run_own(state):
    import q8_block_quantized_gemv_gb300 as q8
    case, op = state["case"], state["op"]
    if op == "slots":
        return q8.kv_slots(state["cached"], state["fresh"], state["table"], state["free"], case["page"],
                           case["capacity"], head=state["head"])
    if "cache" not in state:  # the handle and the workspace that a program keeps
        if op == "append":
            state["cache"] = q8.KVCache(state["k_cache"], state["v_cache"])
        else:
            state["cache"] = q8.KVCache(state["k"], state["v"], state.get("k_scale"), state.get("v_scale"))
            state["workspace"] = q8.attn_workspace()
    if op == "append":
        q = q8.rope_append(state["q"], state["k"], state["v"], state["cache"], state["positions"], state["slots"],
                           table=state["table"], interleaved=case["interleaved"], q_gamma=state["q_gamma"],
                           k_gamma=state["k_gamma"], eps=1e-6)
        return q, state["k_cache"], state["v_cache"]
    if op == "decode":
        return q8.attn_decode(state["q"], state["cache"], state["table"], state["lens"], scale=state["scale"],
                              window=case["window"], sinks=case["sinks"], workspace=state["workspace"])
    return q8.attn_prefill(state["q"], state["cache"], state["table"], state["lens"], state["row_start"],
                           scale=state["scale"], window=case["window"], sinks=case["sinks"],
                           workspace=state["workspace"])


def _plain_slots(state):
    case, page = state["case"], state["case"]["page"]
    cached, fresh, table, free, head = (state[k] for k in ("cached", "fresh", "table", "free", "head"))
    width, capacity = table.shape[1], case["capacity"]
    lens = cached + fresh
    have = (cached + page - 1) // page
    want = torch.clamp((lens + page - 1) // page, max=width)
    need = torch.clamp(want - have, min=0)
    ends = torch.cumsum(need, 0)
    col = torch.arange(width, device=table.device)[None, :]
    index = head + (ends - need)[:, None] + col - have[:, None]
    new = (col >= have[:, None]) & (col < want[:, None])
    taken = torch.where(index < free.numel(), free[torch.clamp(index, 0, free.numel() - 1)], -1)
    table.copy_(torch.where(new, taken, table))
    row_end = torch.cumsum(fresh, 0)
    row_start = torch.cat([torch.zeros_like(row_end[:1]), row_end])
    row = torch.arange(capacity, device=table.device)
    r = torch.clamp(torch.searchsorted(row_end, row, right=True), max=fresh.numel() - 1)
    live = row < row_end[-1]
    pos = torch.where(live, cached[r] + row - row_start[r], -1)
    at = torch.clamp(pos, min=0)
    entry = torch.where(at // page < width, table[r, torch.clamp(at // page, max=width - 1)], -1)
    slots = torch.where(live & (entry >= 0), entry.to(torch.int64) * page + at % page, -1)
    return {"table": table, "lens": lens, "row_start": row_start.to(torch.int32), "positions": pos.to(torch.int32),
            "slots": slots, "head": (head + ends[-1:]).to(torch.int32)}


def _rotated(x, gamma, state, cos, sin):
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma
    n = state["case"]["rotary"]
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if state["case"]["interleaved"] else (x[..., : n // 2], x[..., n // 2: n])
    c, d = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([c, d], -1).flatten(-2) if state["case"]["interleaved"] else torch.cat([c, d], -1)
    return torch.cat([turned, x[..., n:]], -1)


def _plain_append(state):
    case = state["case"]
    rows, dim, page, half = case["rows"], case["dim"], case["page"], case["rotary"] // 2
    pos, slots = state["positions"], state["slots"]
    turn = state["table"][torch.clamp(pos, min=0).long()][:, None, :]
    cos, sin = turn[..., :half], turn[..., half:]
    q = _rotated(state["q"].view(rows, case["heads"], dim), state["q_gamma"], state, cos, sin)
    k = _rotated(state["k"].view(rows, case["kv_heads"], dim), state["k_gamma"], state, cos, sin)
    v = state["v"].view(rows, case["kv_heads"], dim)
    live = (pos >= 0)[:, None, None]
    q = torch.where(live, q, 0.0).to(torch.bfloat16).view(rows, -1)
    # a row without a slot writes nothing: it repeats the first row's write (row 0 always holds a token)
    src = torch.where(slots >= 0, torch.arange(rows, device=slots.device), 0)
    to = slots[src]
    for name, x in (("k_cache", k), ("v_cache", v)):
        state[name][to // page, :, to % page] = x.to(torch.bfloat16)[src]
    return q, state["k_cache"], state["v_cache"]


def _gathered(state, name):
    """The pages of every request, in order, as fp32 [requests, kv_heads, width * page, dim]."""
    table = state["table"].clamp(min=0).long()
    x = state[name][table]  # [requests, width, kv_heads, page, dim]
    if state["case"]["cache"] == "q8":
        shape = x.shape
        d = state[name + "_scale"][table]
        x = (x.view(*shape[:-1], -1, BLOCK).float() * d[..., None]).view(shape)
    r, w, h, p, dim = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(r, h, w * p, dim).float()


def _attend(q, k, v, seen, scale):
    """q [r, h, n, dim], k and v [r, h, len, dim], seen [r, 1, n, len] -> fp32 [r, h, n, dim]; 0 where nothing is seen."""
    s = (q * scale) @ k.transpose(-1, -2)
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, (p @ v) / total, 0.0)


def _seen(state, pos, lens, length):
    """Which of `length` keys the rows at positions pos [r, n] see -> [r, 1, n, length]."""
    case = state["case"]
    key = torch.arange(length, device=pos.device)[None, None, :]
    at = pos[:, :, None]
    seen = (key <= at) & (key < lens[:, None, None])
    if case["window"]:
        seen = seen & ((at - key < case["window"]) | (key < case["sinks"]))
    return seen[:, None]


def _plain_decode(state):
    case = state["case"]
    k, v = _gathered(state, "k"), _gathered(state, "v")
    n = case["heads"] // case["kv_heads"]
    q = state["q"].float().view(case["requests"], case["kv_heads"], n, case["dim"])
    seen = _seen(state, state["lens"][:, None] - 1, state["lens"], k.shape[2])
    return _attend(q, k, v, seen, state["scale"]).to(torch.bfloat16).view(case["requests"], -1)


def _plain_prefill(state):
    case = state["case"]
    lens, start, most = state["lens"], state["row_start"], state["most"]
    r, h, dim = case["requests"], case["kv_heads"], case["dim"]
    n = case["heads"] // h
    k, v = _gathered(state, "k"), _gathered(state, "v")
    fresh = start[1:] - start[:-1]
    step = torch.arange(most, device=lens.device)[None, :]
    index = torch.clamp(start[:-1, None] + step, max=case["rows"] - 1).long()
    q = state["q"].float()[index].view(r, most, h, n, dim).permute(0, 2, 3, 1, 4).reshape(r, h, n * most, dim)
    pos = (lens - fresh)[:, None] + step
    seen = _seen(state, pos, lens, k.shape[2]).repeat(1, 1, n, 1)
    out = _attend(q, k, v, seen, state["scale"]).to(torch.bfloat16)
    out = out.view(r, h, n, most, dim).permute(0, 3, 1, 2, 4).reshape(r, most, h * n * dim)
    row = torch.arange(case["rows"], device=lens.device, dtype=torch.int32)
    of = torch.searchsorted(start[1:].contiguous(), row, right=True)
    return out[of, row - start[of]]


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def _visible(first, count, window, sinks):
    """Visible (query, key) pairs of `count` queries from position `first` on, and the keys that any of them sees."""
    if not window:
        return count * first + count * (count + 1) // 2, first + count
    pairs = 0
    for p in range(first, first + count):
        low = max(0, p - window + 1)
        pairs += p + 1 - low + min(sinks, low)
    low = max(0, first - window + 1)
    return pairs, (first + count - low + min(sinks, low)) if count else 0


def work(case):
    if case["op"] == "append":
        n = case["heads"] + 2 * case["kv_heads"]
        rows = case["rows"]
        norms = 2 * case["dim"] * 4 if case["norm"] else 0
        return {"bytes": rows * (n * case["dim"] * 6 + case["rotary"] * 4 + 12) + norms,
                "flops": rows * (case["heads"] + case["kv_heads"]) * (3 * case["rotary"] + 4 * case["dim"] * case["norm"])}
    cached, fresh = _requests(case)
    if case["op"] == "slots":
        new = sum(_pages_of(c + f, case["page"]) - _pages_of(c, case["page"]) for c, f in zip(cached, fresh))
        return {"bytes": len(cached) * 16 + 8 + new * 8 + case["capacity"] * 12, "flops": 0}
    value = 2.0 if case["cache"] == "bf16" else 1.125
    pairs = keys = 0
    for c, f in zip(cached, fresh):
        p, k = _visible(c, f, case["window"], case["sinks"])
        pairs, keys = pairs + p, keys + k
    rows = len(cached) if case["op"] == "decode" else case["rows"]
    moved = keys * case["kv_heads"] * case["dim"] * 2 * value + rows * case["heads"] * case["dim"] * 4
    return {"bytes": int(moved) + len(cached) * 8, "flops": pairs * case["heads"] * case["dim"] * 4}


# ---- the definition, in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers
    state = prepare(case, seed)
    dim, heads, kv_heads, page = case["dim"], case["heads"], case["kv_heads"], case["page"]
    if case["op"] == "append":
        out = {"q": torch.zeros(case["rows"], heads, dim, dtype=torch.float64, device="cuda"),
               "k": state["k_cache"].double(), "v": state["v_cache"].double()}
        live = torch.nonzero(state["positions"] >= 0).flatten()
        turn = torch.complex(*(x.double() for x in state["table"][state["positions"][live].long()].chunk(2, 1)))[:, None]
        slot = state["slots"][live]
        for name, n in (("q", heads), ("k", kv_heads), ("v", kv_heads)):
            x = state[name].double().view(case["rows"], n, dim)[live]
            if name != "v":
                if case["norm"]:
                    x = x / ((x ** 2).sum(-1, keepdim=True) / dim + 1e-6).sqrt() * state[name + "_gamma"].double()
                m = case["rotary"]
                pair = x[..., :m].unflatten(-1, (m // 2, 2) if case["interleaved"] else (2, m // 2))
                pair = pair if case["interleaved"] else pair.transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
                z = z if case["interleaved"] else z.transpose(-1, -2)
                x = torch.cat([z.flatten(-2), x[..., m:]], -1)
            if name == "q":
                out["q"][live] = x
            else:
                out[name][slot // page, :, slot % page] = x
        return out["q"].view(case["rows"], -1), out["k"], out["v"]
    cached, fresh = _requests(case)
    rows = len(cached) if case["op"] == "decode" else case["rows"]
    out = torch.zeros(rows, heads, dim, dtype=torch.float64, device="cuda")
    q = state["q"].double().view(rows, heads, dim)
    row = 0
    for i, (c, f) in enumerate(zip(cached, fresh)):
        if not f:
            row += case["op"] == "decode"
            continue
        pages = state["table"][i, : _pages_of(c + f, page)].long()
        at = torch.arange(c, c + f, device="cuda")[:, None]
        for h in range(kv_heads):
            kv = {}
            for name in ("k", "v"):
                x = state[name][pages, h].double()
                if case["cache"] == "q8":
                    x = x * state[name + "_scale"][pages, h].double().repeat_interleave(BLOCK, -1)
                kv[name] = x.reshape(-1, dim)[: c + f]
            key = torch.arange(c + f, device="cuda")[None, :]
            hidden = key > at
            if case["window"]:
                hidden |= (at - key >= case["window"]) & (key >= case["sinks"])
            for g in range(heads // kv_heads):
                head = h * (heads // kv_heads) + g
                w = (q[row: row + f, head] @ kv["k"].T * state["scale"]).masked_fill(hidden, -math.inf).softmax(-1)
                out[row: row + f, head] = w @ kv["v"]
        row += f
    return out.view(rows, -1)
