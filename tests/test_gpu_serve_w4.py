"""The example's serving loop over 4-bit weights and with rules on the logits: every operator together, against a plain 64-bit
decoder over the whole sequences and the rules written out in 64 bits."""
import pytest
import torch

from test_gpu_serve import plain_logits, serve, tolerance  # noqa: F401

pytestmark = pytest.mark.gpu


def model(serve, layers=2, vocab=999, weights="q4", positions=512):
    return serve.Model(layers=layers, width=256, heads=4, kv_heads=2, dim=64, ffn=448, vocab=vocab, positions=positions, seed=5,
                       weights=weights)


@pytest.mark.parametrize("cache,window", [("bf16", 0), ("q8", 100)])
def test_served_logits_are_the_plain_decoders(serve, cache, window):
    """The products are of the bf16 rows and the exact weights, so that a layer's roundings are those over Q8_0 weights."""
    layers, steps = 2, 4
    lengths = (1, 37, 130, 470)  # 638 rows: two prefill steps, of more than 16 rows; the decoding's have four
    m = model(serve, layers)
    server = serve.Server(m, len(lengths), sum(-(-(n + steps) // 32) for n in lengths), 32, cache, window)
    g = torch.Generator().manual_seed(6)
    prompts = [torch.randint(m.vocab, (n,), generator=g).tolist() for n in lengths]
    said = [server.prefill(prompts)]
    logits = [server.logits.clone()]
    for _ in range(steps):
        said.append(server.decode(1)[0].clone())
        logits.append(server.logits.clone())
    for r, prompt in enumerate(prompts):
        tokens = prompt + [t[r].item() for t in said[:-1]]
        want = plain_logits(m, tokens, serve.EPS, window, 0)[-(steps + 1):]
        got = torch.stack([x[r, :m.vocab] for x in logits]).double()
        err = ((got - want).norm(dim=1) / want.norm(dim=1)).max().item()
        assert err <= tolerance(layers), f"request {r}: {err}"
        for x, t in zip(got, said):  # no rules: the first maximum
            assert x.argmax().item() == t[r].item()
    assert serve.q8.device_fault() == 0


def ruled(rules, logits, prompt, answer):
    """The rules in 64 bits on one row of logits: the values among which the choice is made."""
    v = logits.double().clone()
    count = torch.zeros_like(v)
    seen = torch.zeros_like(v, dtype=torch.bool)
    seen[prompt + answer] = True
    for t in answer:
        count[t] += 1
    v = torch.where(seen, torch.where(v > 0, v / rules.repetition, v * rules.repetition), v)
    v -= rules.frequency * count + rules.presence * (count > 0)
    for t, b in rules.bias.items():
        v[t] += b
    if rules.temperature > 0:
        v /= rules.temperature
    return v if rules.allowed is None else v.masked_fill(~rules.allowed.to(v.device), -float("inf"))


@pytest.mark.parametrize("weights", ["q4", "q8"])
@pytest.mark.parametrize("temperature", [0.0, 0.7])
def test_every_token_follows_the_rules(serve, weights, temperature):
    """Through prefill steps, captured decoding, and a second turn of the conversation.  The kernel's fp32 values are off by
    at most a rounding for each of six rules, relative to what passes through them."""
    m = model(serve, 1, 200, weights)
    rules = serve.Rules(1.3, 0.25, 0.5, temperature, bias={7: 3.0, 11: -2.5, 60: 1.5}, allowed=torch.arange(200) % 5 != 3)
    lengths, steps = (3, 300, 400), 12  # the prompts take two steps
    server = serve.Server(m, 3, 64, 32, rules=rules)
    g = torch.Generator().manual_seed(7)
    before, answer = [[] for _ in lengths], [[] for _ in lengths]

    def told(tokens):
        for r in range(len(lengths)):
            v = ruled(rules, server.logits[r, :m.vocab], before[r], answer[r])
            if temperature > 0:
                v = v + server.rules["noise"][r].double()
            t = tokens[r].item()
            assert rules.allowed[t] and v[t] >= v.max() - 16 * 2.0 ** -24 * (v[v > -1e30].abs().max() + 10)
            answer[r].append(t)

    for turn in range(2):
        prompts = [torch.randint(m.vocab, (n if turn == 0 else 5,), generator=g).tolist() for n in lengths]
        for r, p in enumerate(prompts):
            before[r] += answer[r][:-1] + p  # the last token told was not fed: the next prompt is in its place
            answer[r] = []
        told(server.prefill(prompts))
        for _ in range(steps):
            told(server.decode(1)[0])
        for r, n in enumerate(lengths):
            assert server.rules["history"][r, :server.rules["lengths"][r]].tolist() == before[r] + answer[r]
    assert any(len(set(a)) > 3 for a in answer)
    assert serve.q8.device_fault() == 0


def test_the_same_seed_says_the_same(serve):
    m = model(serve, 1, 200)
    said = []
    for seed in (3, 3, 4):
        server = serve.Server(m, 2, 16, 32, rules=serve.Rules(temperature=2.0, seed=seed))
        said.append([server.prefill([[5, 6], [7]]).tolist(), server.decode(10).tolist()])
    assert said[0] == said[1] != said[2]


def test_the_command_runs(serve, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["serve.py", "--requests", "3", "--prompt", "70", "--tokens", "4", "--layers", "1",
                                     "--weights", "q4", "--repetition", "1.2", "--temperature", "0.8"])
    serve.main()
    out = capsys.readouterr().out
    assert "prefill: 189 tokens of 3 prompts" in out and "decode: 2 steps of 3 requests" in out
