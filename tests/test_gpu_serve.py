"""The example's serving loop, every operator together, against a plain 64-bit decoder over the whole sequences."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def serve():
    spec = importlib.util.spec_from_file_location("serve_example", os.path.join(ROOT, "examples", "serve.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def norm(x, gamma, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * gamma.double()


def rotate(x, table):
    """x [tokens, heads, dim], halves rotated over the table's width."""
    rot = table.shape[1]
    c, s = (t.double()[:x.shape[0], None] for t in table.split(rot // 2, 1))
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., rot:]], -1)


def plain_logits(m, tokens, eps, window, sinks):
    n = len(tokens)
    h = m.embedding[torch.tensor(tokens, device="cuda")].double()
    x = norm(h, m.first_norm, eps)
    i, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")[None, :]
    seen = (j <= i) & ((i - j < window) | (j < sinks) if window else True)
    for w in m.layers:
        q, k, v = ((x @ w[t].dense()).view(n, -1, m.dim) for t in "qkv")
        q, k = rotate(norm(q, w["q_norm"], eps), m.rope), rotate(norm(k, w["k_norm"], eps), m.rope)
        k, v = (t.repeat_interleave(m.heads // m.kv_heads, 1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) * m.dim ** -0.5
        p = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
        a = torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1)
        h = h + a @ w["o"].dense()
        x = norm(h, w["mid_norm"], eps)
        g, u = x @ w["gate"].dense(), x @ w["up"].dense()
        h = h + (torch.nn.functional.silu(g) * u) @ w["down"].dense()
        x = norm(h, w["next_norm"], eps)
    return x @ m.head.dense()


# A layer rounds seven things on the way to its outputs to bf16 or, in a quantized cache, to about as much: the normed
# rows (twice), q, the cached keys and values, the weights, the attention's output and the gated pair's; the roundings of
# q and k move scores of a few units, which counts each of them three times more.  With the last norm that is 13 roundings
# of at most 2^-8 a layer and one more, of rows that the products carry on without growing them.
def tolerance(layers):
    return (13 * layers + 1) * 2.0 ** -8


@pytest.mark.parametrize("cache,dim,heads,kv_heads,page,window,sinks,rotary", [
    ("bf16", 128, 4, 4, 16, 0, 0, None),
    ("bf16", 64, 6, 2, 48, 40, 3, 32),
    ("q8", 128, 8, 2, 32, 0, 0, None),
    ("q8", 64, 4, 1, 16, 100, 0, None),
])
def test_served_logits_are_the_plain_decoders(serve, cache, dim, heads, kv_heads, page, window, sinks, rotary):
    layers, steps = 2, 5
    lengths = (1, 37, 130, 470)  # 638 rows: two prefill steps
    m = serve.Model(layers=layers, width=256, heads=heads, kv_heads=kv_heads, dim=dim, ffn=416, vocab=999,
                    positions=512, rotary=rotary, seed=5)
    pages = sum(-(-(n + steps) // page) for n in lengths)
    server = serve.Server(m, len(lengths), pages, page, cache, window, sinks)
    g = torch.Generator().manual_seed(6)
    prompts = [torch.randint(m.vocab, (n,), generator=g).tolist() for n in lengths]
    first = server.prefill(prompts)
    logits = [server.logits.clone()]
    said = [first]
    for _ in range(steps):
        said.append(server.decode(1)[0].clone())
        logits.append(server.logits.clone())
    torch.cuda.synchronize()
    assert server.cached.tolist() == [n + steps for n in lengths]
    for r, prompt in enumerate(prompts):
        tokens = prompt + [t[r].item() for t in said[:-1]]
        want = plain_logits(m, tokens, serve.EPS, window, sinks)[-(steps + 1):]
        got = torch.stack([x[r, :m.vocab] for x in logits]).double()
        err = ((got - want).norm(dim=1) / want.norm(dim=1)).max().item()
        assert err <= tolerance(layers), f"request {r}: {err}"
        for x, t in zip(got, said):  # the first maximum of the logits
            assert x.argmax().item() == t[r].item()
    assert serve.q8.device_fault() == 0


def test_the_command_runs(serve, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["serve.py", "--requests", "3", "--prompt", "70", "--tokens", "4", "--layers", "1",
                                     "--cache", "q8"])
    serve.main()
    out = capsys.readouterr().out
    assert "prefill: 189 tokens of 3 prompts" in out and "decode: 2 steps of 3 requests" in out


def test_what_a_server_refuses(serve):
    """More requests than a step has rows (their last rows would never come together), prompts without a token (whose last
    row is another's), more tokens than pages or positions."""
    m = serve.Model(layers=1, width=256, heads=2, kv_heads=1, dim=64, ffn=416, vocab=99, positions=40, seed=5)
    for requests in (0, serve.CHUNK + 1):
        with pytest.raises(ValueError):
            serve.Server(m, requests, 8, 16)
    server = serve.Server(m, 2, 4, 16)
    for prompts in ([[1]], [[1], []], [[1], [2], [3]], [[1] * 41, [2]], [[1] * 33, [2] * 17]):
        with pytest.raises(ValueError):
            server.prefill(prompts)
    first = server.prefill([[1] * 30, [2] * 3])
    assert server.cached.tolist() == [30, 3] and first.numel() == 2
    server.decode(10)
    with pytest.raises(ValueError):  # the 41st position
        server.decode(1)
    assert server.cached.tolist() == [40, 13] and torch.isfinite(server.logits[:, :99]).all()


def test_as_many_requests_as_a_step_has_rows(serve):
    m = serve.Model(layers=1, width=256, heads=2, kv_heads=1, dim=64, ffn=416, vocab=99, positions=40, seed=5)
    server = serve.Server(m, serve.CHUNK, 2 * serve.CHUNK, 16)
    prompts = [[r % 99] * (1 + r % 3) for r in range(serve.CHUNK)]
    server.prefill(prompts)
    server.decode(2)
    assert server.cached.tolist() == [len(p) + 2 for p in prompts]
