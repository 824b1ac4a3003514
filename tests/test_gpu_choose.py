"""The rules on logits and the token chosen, on the GPU.  Every step is one fp32 operation that rounds once, so that numpy's
fp32 arithmetic gives the same bits; the choice is then a first maximum."""
import numpy as np
import pytest
import torch

import q8_block_quantized_gemv_gb300 as q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_block_quantized_gemv_gb300 import build
    build.build()


def expected(logits, N, repetition=None, frequency=None, presence=None, temperature=None, history=None, lengths=None,
             prompts=None, bias_ids=None, bias=None, mask=None, mask_rows=None, noise=None):
    """Row by row from the description, numpy arrays in and out."""
    m = logits.shape[0]
    out, idx = logits[:, :N].copy(), np.full(m, -1, dtype=np.int64)
    f = np.float32
    with np.errstate(all="ignore"):
        for r in range(m):
            v = out[r]
            if history is not None:
                n = min(max(int(lengths[r]), 0), history.shape[1])
                p = min(max(int(prompts[r]), 0), n) if prompts is not None else 0
                said, seen = history[r, p:n], history[r, :n]
                said, seen = said[(said >= 0) & (said < N)], seen[(seen >= 0) & (seen < N)]
                count = np.bincount(said, minlength=N).astype(f)
                was = np.bincount(seen, minlength=N) > 0
                if repetition is not None:
                    v = np.where(was, np.where(v > 0, v / repetition[r], v * repetition[r]), v).astype(f)
                if frequency is not None:
                    v = np.where(count > 0, v - frequency[r] * count, v).astype(f)
                if presence is not None:
                    v = np.where(count > 0, v - presence[r], v).astype(f)
            if bias_ids is not None:
                add = {int(i): b for i, b in zip(bias_ids[r], bias[r]) if 0 <= i < N}
                for i, b in add.items():
                    v[i] = v[i] + b
            hot = temperature is not None and temperature[r] > 0
            if hot:
                v = (v / temperature[r]).astype(f)
            allowed = np.ones(N, dtype=bool)
            k = r if mask_rows is None else int(mask_rows[r])
            if mask is not None and 0 <= k < mask.shape[0]:
                bits = np.unpackbits(np.ascontiguousarray(mask[k]).view(np.uint8), bitorder="little")
                allowed = bits[:N].astype(bool)
            score = (v + noise[r, :N]).astype(f) if noise is not None and hot else v
            if allowed.any():
                at = np.flatnonzero(allowed)
                s = score[at]
                idx[r] = at[np.flatnonzero(np.isnan(s))[0] if np.isnan(s).any() else np.argmax(s)]
            out[r] = np.where(allowed, v, f(-np.inf))
    return out, idx


def same(a, b):
    return np.array_equal(a.view(np.uint32)[~np.isnan(a)], b.view(np.uint32)[~np.isnan(b)]) and \
        np.array_equal(np.isnan(a), np.isnan(b))


def run(logits, N=None, place=False, **rules):
    """The library's answer against `expected`, bit for bit; what is not a rule's tensor is passed through."""
    N = logits.shape[1] if N is None else N
    want, first = expected(logits, N, **rules)
    dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in rules.items()}
    x = torch.from_numpy(logits).cuda()
    out = x if place else torch.full(x.shape, 77.0, device="cuda")
    idx = q8.choose(x, N, out=out, **dev)
    got = out.cpu().numpy()
    assert same(got[:, :N].copy(), want), "the logits differ"
    assert np.array_equal(idx.cpu().numpy(), first), "the tokens differ"
    if not place:
        assert (got[:, N:] == 77).all()
        assert np.array_equal(x.cpu().numpy().view(np.uint32), logits.view(np.uint32))
        assert torch.equal(q8.choose(x, N, **dev), idx)
    return got, first


def everything(m, N, width, seed, count=5, wide=False, low=0):
    g = np.random.default_rng(seed)
    f = np.float32
    lengths = g.integers(0, width + 1, m).astype(np.int32)
    lengths[0] = width
    words = (N + 31) // 32
    mask = g.integers(-2 ** 31, 2 ** 31, (3, words)).astype(np.int32)
    return {"repetition": (0.7 + g.random(m)).astype(f), "frequency": g.standard_normal(m).astype(f),
            "presence": g.standard_normal(m).astype(f),
            "temperature": np.where(np.arange(m) % 3 == 2, 0, 0.3 + g.random(m)).astype(f),
            "history": (low + N * g.random((m, width)) ** 3).astype(np.int64 if wide else np.int32).clip(low, N - 1),
            "lengths": lengths, "prompts": (lengths // 2).astype(np.int32),
            "bias_ids": np.stack([g.permutation(max(N, count))[:count] for _ in range(m)]).astype(np.int32),
            "bias": (5 * g.standard_normal((m, count))).astype(f), "mask": mask,
            "mask_rows": g.integers(-1, 4, m).astype(np.int32), "noise": g.gumbel(size=(m, N)).astype(f)}


def logits_of(m, N, seed, pitch=None):
    x = np.random.default_rng(seed).standard_normal((m, pitch or N)).astype(np.float32) * 4
    return x


@pytest.mark.parametrize("m,N", [(1, 1), (1, 31), (2, 32), (3, 33), (5, 1000), (1, 4097), (16, 32000), (7, 32003),
                                 (2, 128256), (40, 5000), (3, 151936), (1, 300001)])
@pytest.mark.parametrize("place", [False, True])
def test_every_rule(m, N, place):
    rules = everything(m, N, 200, seed=m + N, wide=N % 2 == 1)
    run(logits_of(m, N, N), place=place, **rules)


RULES = ("repetition", "frequency", "presence", "temperature", "bias_ids", "mask", "noise", "prompts")


@pytest.mark.parametrize("name", RULES)
@pytest.mark.parametrize("alone", [False, True])
def test_each_rule_alone_and_left_out(name, alone):
    m, N = 6, 1030
    rules = everything(m, N, 77, seed=5)
    with_ = {"bias_ids": ("bias",), "mask": ("mask_rows",)}.get(name, ())
    if alone:
        need = ("history", "lengths") if name in ("repetition", "frequency", "presence", "prompts") else \
            ("temperature",) if name == "noise" else ()
        rules = {k: v for k, v in rules.items() if k == name or k in with_ + need}
    else:
        rules = {k: v for k, v in rules.items() if k != name and k not in with_}
    run(logits_of(m, N, 6), **rules)


def test_no_rules_is_the_first_maximum():
    x = np.float32([[1, 3, 3, 2], [-1, -1, -2, -1], [-0.0, 0.0, -1, 0], [np.nan, 5, np.nan, 1], [1, np.inf, np.inf, 0],
                    [-np.inf] * 4])
    _, idx = run(x)
    assert idx.tolist() == [1, 0, 0, 0, 1, 0]


@pytest.mark.parametrize("N", [40, 5000])
def test_rows_that_allow_nothing_or_one_token(N):
    """Hidden tokens are not looked at, whatever they hold; -inf among the allowed is still a token."""
    x = logits_of(5, N, 8)
    x[:, 3] = np.nan
    x[:, 9] = np.inf
    x[4, :] = -np.inf
    mask = np.zeros((5, (N + 31) // 32), dtype=np.int32)
    mask[1, 0], mask[2, -1], mask[4, 1] = 1 << 7, 1 << ((N - 1) % 32), 1 << 4
    mask[0, -1] = 0 if N % 32 == 0 else -1 << (N % 32)  # bits past the vocabulary say nothing
    _, idx = run(x, mask=mask)
    assert idx.tolist() == [-1, 7, N - 1, -1, 36]


def test_logits_of_any_kind():
    """Infinities, NaN, zeros of both signs and the type's lowest value through every rule."""
    m, N = 4, 999
    x = logits_of(m, N, 9)
    special = np.float32([np.inf, -np.inf, np.nan, 0.0, -0.0, np.finfo(np.float32).min, np.finfo(np.float32).max, 1e-45])
    for i, s in enumerate(special):
        x[:, i * 7::61] = s
    rules = everything(m, N, 300, seed=10)
    run(x, **rules)
    rules["temperature"][:] = [-1.0, np.nan, np.inf, 1e-30]
    rules["repetition"][:] = [1.0, 1e30, 1e-30, 1.5]
    rules["frequency"][0], rules["presence"][1] = np.inf, 3e38
    run(x, **rules)


def test_quotients_are_rounded_once():
    """Logits over temperatures of every kind, those just below a power of two among them, bit for bit the division's."""
    m, N = 64, 40000
    g = np.random.default_rng(30)
    t = np.exp2(g.uniform(-3, 3, m)).astype(np.float32)
    t[:8] = np.nextafter(np.exp2(np.arange(-4, 4)).astype(np.float32), np.float32(0))
    t[8:16] = np.nextafter(np.exp2(np.arange(-4, 4)).astype(np.float32), np.float32(np.inf))
    t[16:22] = [1.0, 2.0 ** -20, 2.0 ** 20, 2.0 ** -21, 2.0 ** 21, 1e-38]
    x = (g.standard_normal((m, N)) * np.exp2(g.integers(-8, 8, (m, N)))).astype(np.float32)
    x[:, ::50] = np.exp2(g.integers(-140, 127, (m, 800))).astype(np.float32)
    x[:, 1::50] = np.nextafter(np.exp2(g.integers(-90, 90, (m, 800))).astype(np.float32), np.float32(0))
    x[:, 2::50] = -x[:, 1::50]
    run(x, temperature=t)


def test_history_of_any_kind():
    """Tokens outside the vocabulary, lengths outside the buffer, a token said many times."""
    m, N, width = 6, 500, 400
    rules = everything(m, N, width, seed=11)
    h = rules["history"]
    h[:, ::5] = -1
    h[:, 1::7] = N
    h[:, 2::9] = 2 ** 31 - 1
    h[1] = 17
    rules["lengths"][:] = [width + 100, width, -3, 0, 1, 2 ** 31 - 1]
    rules["prompts"][:] = [5, 0, 9, 2 ** 31 - 1, -7, 399]
    run(logits_of(m, N, 12), **rules)
    wide = dict(rules, history=h.astype(np.int64))
    wide["history"][0, 3], wide["history"][0, 4] = 2 ** 32 + 5, -2 ** 40 + 6
    run(logits_of(m, N, 12), **wide)


def test_long_history():
    m, N, width = 2, 2000, 131073
    rules = everything(m, N, width, seed=13)
    rules["history"][1, :100000] = 3
    run(logits_of(m, N, 14), **rules)


def test_the_longest_history():
    width = 1048575
    history = np.full((1, width), 5, dtype=np.int32)
    lengths = np.int32([width])
    run(logits_of(1, 64, 15), history=history, lengths=lengths, frequency=np.float32([1e-3]))


@pytest.mark.parametrize("N,width", [(500000, 20000), (393217, 8193), (131072, 8193)])
def test_a_long_history_over_a_wide_vocabulary(N, width):
    rules = everything(2, N, width, seed=18)
    rules["history"][0, ::3] = N - 1
    run(logits_of(2, N, 19), **rules)


@pytest.mark.parametrize("count", [1, 300, 2047])
def test_biases(count):
    m, N = 3, 4000
    g = np.random.default_rng(16)
    ids = g.integers(-2, N + 2, (m, count)).astype(np.int32)  # the same token twice: the last one counts
    ids[0, :] = 1234
    run(logits_of(m, N, 17), bias_ids=ids, bias=g.standard_normal((m, count)).astype(np.float32) * 9)


def test_ties_go_to_the_lowest():
    m, N = 3, 70000
    x = np.zeros((m, N), dtype=np.float32)
    x[1, 60000:] = 2
    x[2, 69999] = 1
    _, idx = run(x)
    assert idx.tolist() == [0, 60000, 69999]


@pytest.mark.parametrize("pitch", [1003, 1024, 1100])
def test_pitches(pitch):
    """The products' padded rows and wider ones; histories and noise that are views."""
    m, N = 5, 1000
    rules = everything(m, N, 50, seed=18)
    x = logits_of(m, N, 19, pitch)
    run(x, N, **rules)
    want, first = expected(x, N, **rules)
    dev = {k: torch.from_numpy(v).cuda() for k, v in rules.items()}
    for name in ("history", "noise", "mask"):
        t = dev[name]
        room = torch.zeros((t.shape[0], t.shape[1] + 5), dtype=t.dtype, device="cuda")
        room[:, 2:2 + t.shape[1]] = t
        dev[name] = room[:, 2:2 + t.shape[1]]
    big = torch.zeros((m, pitch + 7), device="cuda")
    big[:, 1:pitch + 1] = torch.from_numpy(x).cuda()
    view = big[:, 1:pitch + 1]
    idx = q8.choose(view, N, out=view, **dev)
    assert same(view[:, :N].cpu().numpy(), want) and np.array_equal(idx.cpu().numpy(), first)
    assert not big[:, 0].any() and not big[:, pitch + 1:].any()


def test_after_a_product_and_in_a_graph():
    """As a decode step ends: logits, rules, choice; captured, replayed over new histories."""
    K, N, m, width = 512, 1001, 4, 64
    g = torch.Generator("cuda").manual_seed(20)
    codes = torch.randint(0, 256, (K // 2, N), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.rand((K // 64, N), device="cuda", generator=g) * 0.02).half()
    w = q8.Weight4(codes, scales)
    x = torch.randn((m, K), device="cuda", generator=g).bfloat16()
    logits = torch.empty((m, w.Np), device="cuda")
    rules = everything(m, N, width, seed=21)
    dev = {k: torch.from_numpy(v).cuda() for k, v in rules.items()}
    idx = torch.empty(m, dtype=torch.int64, device="cuda")

    def step():
        q8.gemv4(x, w, y=logits, constant_weights=True)
        q8.choose(logits, N, out=logits, idx=idx, **dev)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (22, 23):
        rules.update(history=everything(m, N, width, seed)["history"], noise=everything(m, N, width, seed)["noise"])
        for k in ("history", "noise"):
            dev[k].copy_(torch.from_numpy(rules[k]))
        x.copy_(torch.randn((m, K), device="cuda", generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        plain = q8.gemv4(x, w).cpu().numpy()
        want, first = expected(plain, N, **rules)
        assert same(logits[:, :N].cpu().numpy(), want) and np.array_equal(idx.cpu().numpy(), first)
        assert not logits[:, N:].any()


def test_on_another_stream():
    m, N = 8, 3000
    rules = everything(m, N, 90, seed=24)
    x = logits_of(m, N, 25)
    want, first = expected(x, N, **rules)
    dev = {k: torch.from_numpy(v).cuda() for k, v in rules.items()}
    logits = torch.from_numpy(x).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty_like(logits)
    side.wait_stream(torch.cuda.current_stream())
    idx = q8.choose(logits, out=out, stream=side, **dev)
    side.synchronize()
    assert same(out.cpu().numpy(), want) and np.array_equal(idx.cpu().numpy(), first)


def test_noise_samples_the_softmax():
    """Gumbel noise: each token comes as often as its probability says (five standard deviations of the count)."""
    m, N = 20000, 40
    row = np.random.default_rng(26).standard_normal(N).astype(np.float32)
    x = torch.from_numpy(np.repeat(row[None], m, 0)).cuda()
    u = torch.rand((m, N), device="cuda", generator=torch.Generator("cuda").manual_seed(27)).clamp(1e-7, 1 - 1e-7)
    t = torch.full((m,), 0.8, device="cuda")
    idx = q8.choose(x, temperature=t, noise=-torch.log(-torch.log(u)))
    got = torch.bincount(idx, minlength=N).cpu().numpy()
    p = np.exp(row.astype(np.float64) / 0.8)
    p /= p.sum()
    assert (np.abs(got - m * p) <= 5 * np.sqrt(m * p * (1 - p)) + 1).all()


def test_what_the_binding_refuses():
    x = torch.zeros((2, 100), device="cuda")
    i32 = {"dtype": torch.int32, "device": "cuda"}
    for kw in (dict(N=101), dict(out=torch.zeros((2, 99), device="cuda")), dict(out=torch.zeros((3, 100), device="cuda")),
               dict(repetition=torch.ones(3, device="cuda")), dict(temperature=torch.ones(2)),
               dict(frequency=torch.ones(2, device="cuda").double()), dict(history=torch.zeros((2, 5), **i32)),
               dict(history=torch.zeros((1, 5), **i32), lengths=torch.zeros(2, **i32)),
               dict(history=torch.zeros((2, 5), device="cuda"), lengths=torch.zeros(2, **i32)),
               dict(bias=torch.zeros((2, 3), device="cuda")), dict(bias_ids=torch.zeros((2, 3), **i32)),
               dict(bias_ids=torch.zeros((2, 3), **i32), bias=torch.zeros((2, 4), device="cuda")),
               dict(mask=torch.zeros((2, 3), **i32)), dict(mask=torch.zeros((2, 4), device="cuda")),
               dict(noise=torch.zeros((2, 50), device="cuda")), dict(idx=torch.zeros(2, **i32)),
               dict(noise=torch.zeros((100, 2), device="cuda").t())):
        with pytest.raises(ValueError):
            q8.choose(x, **kw)
    with pytest.raises(ValueError):
        q8.choose(torch.zeros((100, 2), device="cuda").t())
    with pytest.raises(q8.Q8Error):
        q8.choose(x, bias_ids=torch.zeros((2, 2048), **i32), bias=torch.zeros((2, 2048), device="cuda"))
    with pytest.raises(q8.Q8Error):  # in place means in place
        big = torch.zeros((2, 300), device="cuda")
        q8.choose(big[:, :100], out=big[:, 50:150])
    assert q8.choose(x[:0]).numel() == 0
