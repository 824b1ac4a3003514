"""A decode step whose weights hold 4 bits, and the choice of its next token, as cases that can be timed.

Four operators, each as a user of the library calls it:

* ``gemv``    the product of a few activation rows (or a prompt's chunk) with a weight of 4-bit codes and group scales,
              or with several such weights of one activation (q/k/v);
* ``glu``     the gated pair over two of them: silu(x.Wg) * (x.Wu), rounded to the next product's bf16;
* ``norm``    the product, the residual add and the next RMS norm;
* ``choose``  penalties for repeated tokens, biases, temperature and grammar masks on the logits, and the token chosen.

A weight is codes 0..15, two to a byte (row 2i in the low half of byte row i), a 16-bit scale for each group of rows of a
column, and a zero point for each group (or 8 for all): value = scale * (code - zero).  With ``own`` false, ``run`` is
elementary torch in fp32; with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False


# ---- the cases -----------------------------------------------------------------------------------------------------

def listed():
    return [
        # One user's attention output projection: a square weight, the finest groups.  Latency.
        {"name": "o_one_user", "op": "gemv", "m": 1, "K": 4096, "widths": "4096", "group": 32, "zeros": False,
         "scales": "fp16"},
        # The q, k and v projections of a full decode batch, 32 query heads over 8, zero points.
        {"name": "qkv_batch", "op": "gemv", "m": 16, "K": 4096, "widths": "4096,1024,1024", "group": 128, "zeros": True,
         "scales": "fp16"},
        # A few users over a width that ends inside a column tile, bf16 scales.
        {"name": "odd_width", "op": "gemv", "m": 5, "K": 5120, "widths": "3000", "group": 64, "zeros": False,
         "scales": "bf16"},
        # One user's logits: the longest stream of weights in a step.
        {"name": "head_one_user", "op": "gemv", "m": 1, "K": 4096, "widths": "128256", "group": 128, "zeros": False,
         "scales": "fp16"},
        # The up projection of the largest prefill chunk: the largest product.
        {"name": "up_chunk", "op": "gemv", "m": 512, "K": 4096, "widths": "14336", "group": 128, "zeros": False,
         "scales": "fp16"},
        # One user's gated pair.
        {"name": "glu_one_user", "op": "glu", "m": 1, "K": 4096, "widths": "14336", "group": 128, "zeros": True,
         "scales": "fp16"},
        # The gated pair of a prompt's last, ragged chunk.
        {"name": "glu_chunk", "op": "glu", "m": 301, "K": 4096, "widths": "14336", "group": 64, "zeros": False,
         "scales": "fp16"},
        # The down projection of a decode batch with the residual and the next layer's norm: a long reduction.
        {"name": "down_batch", "op": "norm", "m": 16, "K": 14336, "widths": "4096", "group": 128, "zeros": True,
         "scales": "fp16"},
        # The output projection of a short prompt in a small model, finest groups.
        {"name": "o_short_prompt", "op": "norm", "m": 61, "K": 2048, "widths": "2048", "group": 32, "zeros": False,
         "scales": "fp16"},
        # One user's next token, greedy under a repetition penalty.  Latency.
        {"name": "choose_one_user", "op": "choose", "m": 1, "N": 32000, "history": 300, "bias": 0, "mask": False,
         "noise": False},
        # A decode batch over a large vocabulary: long conversations, biases, some rows under a grammar.
        {"name": "choose_batch", "op": "choose", "m": 16, "N": 128256, "history": 8191, "bias": 20, "mask": True,
         "noise": True},
        # A large server's step.
        {"name": "choose_large", "op": "choose", "m": 256, "N": 128256, "history": 2001, "bias": 300, "mask": True,
         "noise": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "glu", "norm", "choose"])
    if op == "choose":
        case = {"op": op, "m": _log_int(rng, 1, 256), "N": _log_int(rng, 1000, 160000),
                "history": _log_int(rng, 1, 16384), "bias": rng.choice([0, 1, 20, 300, 2000]),
                "mask": rng.random() < 0.5, "noise": rng.random() < 0.5}
        # at most the tokens of the largest listed step, in the logits and in the histories
        case["m"] = max(1, min(case["m"], 256 * 128256 // case["N"], 256 * 2001 // case["history"]))
        case["bias"] = min(case["bias"], 256 * 300 // case["m"])
        return case
    group = rng.choice([32, 64, 128])
    case = {"op": op, "m": _log_int(rng, 1, 512), "K": max(1, _log_int(rng, 256, 14336) // group) * group, "group": group,
            "zeros": rng.random() < 0.5, "scales": rng.choice(["fp16", "fp16", "bf16"])}
    # at most the products and the bytes of the largest listed chunk
    most = min(16384, 512 * 4096 * 14336 // (case["m"] * case["K"] * (2 if op == "glu" else 1)))
    case["widths"] = str(_log_int(rng, 40, most))
    if op == "gemv" and rng.random() < 0.3:
        n = int(case["widths"])
        case["widths"] = "%d,%d,%d" % (n // 2 + 1, n // 5 + 1, n // 5 + 1)
    return case


def _widths(case):
    return [int(n) for n in case["widths"].split(",")] * (2 if case["op"] == "glu" else 1)


def _padded(n):
    return (n + 31) // 32 * 32  # outputs are whole 32-column tiles, the last one's padding zero


# ---- what a program has in hand before the call --------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + case["m"])
    state = {"case": case}
    if case["op"] == "choose":
        state.update(_prepare_choose(case, gen, random.Random(seed * 31 + case["N"])))
        return state
    m, K, G = case["m"], case["K"], case["group"]
    x = torch.randn((m, K), generator=gen, device="cuda")
    x[:, :: max(1, K // 7)] *= 8.0  # a few strong channels
    state["x"] = x.to(torch.bfloat16)
    state["weights"] = []
    kind = torch.float16 if case["scales"] == "fp16" else torch.bfloat16
    for n in _widths(case):
        codes = torch.randint(0, 256, (K // 2, n), generator=gen, device="cuda", dtype=torch.uint8)
        scales = ((0.5 + torch.rand((K // G, n), generator=gen, device="cuda")) * (0.2 / math.sqrt(K))).to(kind)
        zeros = None
        if case["zeros"]:
            zeros = torch.randint(5, 12, (K // G, n), generator=gen, device="cuda", dtype=torch.uint8)
        state["weights"].append((codes, scales, zeros))
    if case["op"] == "norm":
        n = _widths(case)[0]
        state["residual"] = torch.zeros((m, _padded(n)), device="cuda")
        state["residual"][:, :n] = torch.randn((m, n), generator=gen, device="cuda")
        state["gamma"] = 0.5 + torch.rand(n, generator=gen, device="cuda")
        state["eps"] = 1e-5
    return state


def _prepare_choose(case, gen, rng):
    m, N = case["m"], case["N"]
    logits = torch.randn((m, N), generator=gen, device="cuda") * 3.0

    def rows(lo, hi):
        return torch.tensor([rng.uniform(lo, hi) for _ in range(m)], device="cuda")

    lengths = [case["history"]] + [rng.randint(0, case["history"]) for _ in range(m - 1)]
    # tokens repeat as in text: few of them often, most of them rarely
    u = torch.rand((m, case["history"]), generator=gen, device="cuda")
    history = (N * u ** 4).to(torch.int32).clamp(max=N - 1)
    state = {"logits": logits, "history": history, "lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda"),
             "prompts": torch.tensor([n // 3 for n in lengths], dtype=torch.int32, device="cuda"),
             "repetition": rows(1.0, 1.3), "frequency": rows(0.0, 0.4), "presence": rows(0.0, 0.6),
             "temperature": None, "bias_ids": None, "bias": None, "mask": None, "mask_rows": None, "noise": None}
    if case["bias"]:
        ids = torch.randint(0, N, (m, case["bias"]), generator=gen, device="cuda", dtype=torch.int32)
        order = torch.sort(ids, dim=1).values  # a token at most once: the others of it are unused places
        order[:, 1:][order[:, 1:] == order[:, :-1]] = -1
        state["bias_ids"] = order
        state["bias"] = torch.randn((m, case["bias"]), generator=gen, device="cuda") * 4.0
    if case["mask"]:  # grammars of a few rows, most rows free; a bit for each token
        count = max(1, m // 4)
        words = (N + 31) // 32
        state["mask"] = torch.randint(-2 ** 31, 2 ** 31, (count, words), generator=gen, device="cuda",
                                      dtype=torch.int64).to(torch.int32)
        state["mask"] &= torch.randint(-2 ** 31, 2 ** 31, (count, words), generator=gen, device="cuda",
                                       dtype=torch.int64).to(torch.int32)
        state["mask_rows"] = torch.tensor([rng.randrange(count) if r % 2 == 0 else -1 for r in range(m)],
                                          dtype=torch.int32, device="cuda")
    if case["noise"]:  # sampling: Gumbel noise on the logits over the temperature; some rows greedy
        u = torch.rand((m, N), generator=gen, device="cuda").clamp_(min=1e-7, max=1 - 1e-7)
        state["noise"] = -torch.log(-torch.log(u))
        state["temperature"] = torch.tensor([0.0 if r % 5 == 4 else rng.uniform(0.5, 1.2) for r in range(m)],
                                            device="cuda")
    return state


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"gemv": _plain_gemv, "glu": _plain_glu, "norm": _plain_norm, "choose": _plain_choose}[state["case"]["op"]](
        state)


def _run_own(state):
    import q8_block_quantized_gemv_gb300 as q8
    op = state["case"]["op"]
    if op == "choose":
        out = torch.empty_like(state["logits"])
        idx = q8.choose(state["logits"], out=out, repetition=state["repetition"], frequency=state["frequency"],
                        presence=state["presence"], temperature=state["temperature"], history=state["history"],
                        lengths=state["lengths"], prompts=state["prompts"], bias_ids=state["bias_ids"],
                        bias=state["bias"], mask=state["mask"], mask_rows=state["mask_rows"], noise=state["noise"])
        return out, idx
    if "w" not in state:  # the weights as a program keeps them, laid out once
        state["w"] = [q8.Weight4(*w) for w in state["weights"]]
    x, w = state["x"], state["w"]
    if op == "glu":
        return q8.gemv4_glu(x, w[0], w[1], want=("bf16",), constant_weights=True)[1]
    if op == "norm":
        return q8.gemv4_residual_norm(x, w[0], state["residual"], state["gamma"], state["eps"], constant_weights=True)
    if len(w) == 1:
        return q8.gemv4(x, w[0], constant_weights=True)
    return q8.gemv4_parts(x, w, constant_weights=True)


def _dense(state, i):
    """The weight's values, fp32 [K, N]."""
    codes, scales, zeros = state["weights"][i]
    group = state["case"]["group"]
    c = torch.stack([codes & 15, codes >> 4], 1).flatten(0, 1).float()
    c = c.view(scales.shape[0], group, -1)
    c = c - (8.0 if zeros is None else zeros.float()[:, None])
    return (c * scales.float()[:, None]).flatten(0, 1)


def _product(state, i):
    y = state["x"].float() @ _dense(state, i)
    return torch.nn.functional.pad(y, (0, _padded(y.shape[1]) - y.shape[1]))


def _plain_gemv(state):
    ys = [_product(state, i) for i in range(len(state["weights"]))]
    return ys[0] if len(ys) == 1 else ys


def _plain_glu(state):
    g, u = _product(state, 0), _product(state, 1)
    return (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)


def _plain_norm(state):
    h = state["residual"] + _product(state, 0)
    n = state["gamma"].numel()
    mean = (h[:, :n] * h[:, :n]).sum(1, keepdim=True) / n
    out = torch.zeros_like(h)
    out[:, :n] = h[:, :n] / torch.sqrt(mean + state["eps"]) * state["gamma"]
    return h, out.to(torch.bfloat16)


def _counts(state):
    """How often each token stands in a row's answer, and whether it stands in the row at all."""
    m, N = state["logits"].shape
    history, at = state["history"], torch.arange(state["history"].shape[1], device="cuda")[None, :]
    live = at < state["lengths"][:, None]
    said = live & (at >= state["prompts"][:, None])
    token = history.long()
    count = torch.zeros((m, N), device="cuda").scatter_add_(1, token, said.float())
    seen = torch.zeros((m, N), device="cuda").scatter_add_(1, token, live.float()) > 0
    return count, seen


def _plain_choose(state):
    v = state["logits"]
    m, N = v.shape
    count, seen = _counts(state)
    rep = state["repetition"][:, None]
    v = torch.where(seen, torch.where(v > 0, v / rep, v * rep), v)
    v = v - state["frequency"][:, None] * count
    v = v - torch.where(count > 0, state["presence"][:, None], 0.0)
    if state["bias"] is not None:
        ids = state["bias_ids"].long()
        v = v.scatter_add(1, ids.clamp(min=0), torch.where(ids >= 0, state["bias"], 0.0))
    if state["temperature"] is not None:
        t = state["temperature"][:, None]
        v = torch.where(t > 0, v / torch.where(t > 0, t, 1.0), v)
    if state["mask"] is not None:
        n = torch.arange(N, device="cuda")
        rows = state["mask_rows"]
        bits = (state["mask"][rows.clamp(min=0).long()][:, n // 32] >> (n % 32).int()) & 1
        v = torch.where((bits != 0) | (rows < 0)[:, None], v, -math.inf)
    score = v
    if state["noise"] is not None:
        score = torch.where(state["temperature"][:, None] > 0, v + state["noise"], v)
    top = score.amax(1, keepdim=True)
    idx = torch.where(score == top, torch.arange(N, device="cuda"), N).amin(1)  # the lowest index among the largest
    return v, idx


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(case):
    m = case["m"]
    if case["op"] == "choose":
        N = case["N"]
        row = N * 8 + case["bias"] * 8 + 24 + (N * 4 if case["noise"] else 0)
        masks = max(1, m // 4) * ((N + 31) // 32) * 4 if case["mask"] else 0
        rng = random.Random(1)  # about the lengths that a seed draws
        tokens = case["history"] + sum(rng.randint(0, case["history"]) for _ in range(m - 1))
        return {"bytes": m * row + masks + tokens * 4, "flops": m * N * 4}
    K, G, widths = case["K"], case["group"], _widths(case)
    weight = sum(K * n // 2 + K // G * n * (3 if case["zeros"] else 2) for n in widths)
    out = sum(_padded(n) for n in widths) * 4
    if case["op"] == "glu":
        out = _padded(widths[0]) * 2
    elif case["op"] == "norm":
        out += _padded(widths[0]) * 6
    return {"bytes": weight + m * K * 2 + m * out, "flops": 2 * m * K * sum(widths)}


# ---- the definition, in 64 bits ------------------------------------------------------------------------------------

def _exact_product(state, i):
    """Group by group: the group's sum of activations times codes, less the zero point's, times its scale."""
    codes, scales, zeros = state["weights"][i]
    G, n = state["case"]["group"], codes.shape[1]
    x = state["x"].double()
    y = torch.zeros((x.shape[0], _padded(n)), dtype=torch.float64, device="cuda")
    for a in range(0, n, 8192):
        b = min(n, a + 8192)
        for k in range(scales.shape[0]):
            byte = codes[k * G // 2: (k + 1) * G // 2, a:b].int()
            xs = x[:, k * G: (k + 1) * G]
            part = xs[:, 0::2] @ (byte % 16).double() + xs[:, 1::2] @ torch.div(byte, 16, rounding_mode="floor").double()
            zero = 8.0 if zeros is None else zeros[k, a:b].double()
            y[:, a:b] += (part - xs.sum(1, keepdim=True) * zero) * scales[k, a:b].double()
    return y


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "choose":
        v = state["logits"].double()
        m, N = v.shape
        lengths, prompts = state["lengths"].tolist(), state["prompts"].tolist()
        for r in range(m):
            tokens = state["history"][r, : lengths[r]].long()
            seen = torch.bincount(tokens, minlength=N)
            count = torch.bincount(tokens[prompts[r]:], minlength=N).double()
            rep = state["repetition"][r].double()
            v[r] = torch.where(seen > 0, v[r].clamp(min=0) / rep + v[r].clamp(max=0) * rep, v[r])
            v[r] -= state["frequency"][r].double() * count + state["presence"][r].double() * count.clamp(max=1)
            if state["bias"] is not None:
                used = state["bias_ids"][r] >= 0
                v[r, state["bias_ids"][r][used].long()] += state["bias"][r][used].double()
            if state["temperature"] is not None and state["temperature"][r] > 0:
                v[r] /= state["temperature"][r].double()
            if state["mask"] is not None and state["mask_rows"][r] >= 0:
                word = state["mask"][state["mask_rows"][r]].long() & 0xFFFFFFFF
                allowed = torch.stack([(word // 2 ** i) % 2 for i in range(32)], 1).flatten()[:N]
                v[r][allowed == 0] = -math.inf
        return v, None  # the tokens chosen are whole numbers
    if case["op"] == "gemv":
        ys = [_exact_product(state, i) for i in range(len(state["weights"]))]
        return ys[0] if len(ys) == 1 else ys
    if case["op"] == "glu":
        g, u = _exact_product(state, 0), _exact_product(state, 1)
        return g * torch.sigmoid(g) * u
    h = state["residual"].double() + _exact_product(state, 0)
    n = state["gamma"].numel()
    out = torch.zeros_like(h)
    out[:, :n] = h[:, :n] * (h[:, :n].square().mean(1, keepdim=True) + state["eps"]).rsqrt() * state["gamma"].double()
    return h, out
