"""Calls with ``stream=`` while the current stream still has work to do on memory that it has already freed: what a call
allocates must not be that memory, and an attention call's own workspace must be zero before its kernel looks."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import q8_block_quantized_gemv_gb300 as q8
    q8.build.build()
    return q8


def leave_work(torch, like):
    """Tensors as large as those of `like`, freed with a write to each still to come."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.empty_like(t) for t in like]
    torch.cuda._sleep(100_000_000)  # some 50 ms
    for t in held:
        t.view(torch.uint8).fill_(0x7B)


def tensors(x):
    if isinstance(x, dict):
        x = x.values()
    if isinstance(x, (list, tuple)) or hasattr(x, "__iter__") and not hasattr(x, "data_ptr"):
        return [t for y in x for t in tensors(y)]
    return [] if x is None else [getattr(x, "buf", x)]


def calls(q8, torch):
    """name -> a call that takes `stream` and returns what it allocates."""
    g = torch.Generator("cuda").manual_seed(3)
    m, K, N = 5, 1024, 2048
    q = torch.randint(-127, 128, (K, N), dtype=torch.int8, device="cuda", generator=g)
    s = torch.rand((K // 32, N), device="cuda", generator=g) * 1e-3
    wide = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    wide_s = torch.rand((N // 32, K), device="cuda", generator=g) * 1e-3
    qt, st = q8.tile_device(q, s, N)
    x = torch.randn((m, K), device="cuda", generator=g).bfloat16()
    h = torch.randn((m, N), device="cuda", generator=g)
    gamma = torch.ones(N, device="cuda")
    heads, dim, page, lens = 8, 128, 16, [3000, 70, 411]
    cache = q8.KVCache.empty(256, 2, page, dim)
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, device="cuda", generator=g))
    table = torch.randperm(3 * 190, device="cuda", generator=g).view(3, 190).remainder(256).int()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lens_d, starts, free = i32(lens), i32([0, 40, 60, 200]), torch.arange(64, dtype=torch.int32, device="cuda")
    qd = torch.randn((3, heads * dim), device="cuda", generator=g).bfloat16()
    qp = torch.randn((200, heads * dim), device="cuda", generator=g).bfloat16()
    xs = [torch.randn((20, n * dim), device="cuda", generator=g) for n in (heads, 2, 2)]
    pos, empty = torch.arange(20, dtype=torch.int32, device="cuda"), q8.KVCache.empty(4, 2, page, dim)
    cached, fresh, paged = i32([0, 5, 31]), i32([17, 1, 1]), torch.full((3, 4), 9, dtype=torch.int32, device="cuda")
    return {
        "quantize_act": lambda stream: q8.quantize_act(x, stream=stream),
        "gemv": lambda stream: q8.gemv(x, q, s, N, stream=stream),
        "gemv_argmax": lambda stream: q8.gemv_argmax(x, qt, st, N, tiled=True, stream=stream),
        "tile_device": lambda stream: q8.tile_device(wide, wide_s, K, stream=stream),
        "gemv_parts": lambda stream: q8.gemv_parts(x, [(qt, st, N), (qt, st, N)], tiled=True, stream=stream),
        "gemv_glu": lambda stream: q8.gemv_glu(x, (qt, st), (qt, st), N, want=("f32", "bf16", "q8"), stream=stream),
        "gemv_residual_norm": lambda stream: q8.gemv_residual_norm(x, qt, st, N, h, gamma, 1e-6, want=("bf16", "q8"),
                                                                    stream=stream),
        "kv_slots": lambda stream: [v for n, v in q8.kv_slots(cached, fresh, paged, free, page, 40, stream=stream).items()
                                    if n != "table"],
        "rope_append": lambda stream: q8.rope_append(*xs, empty, pos, pos.long(), stream=stream),
        "attn_decode": lambda stream: q8.attn_decode(qd, cache, table, lens_d, stream=stream),
        "attn_prefill": lambda stream: q8.attn_prefill(qp, cache, table, lens_d, starts, stream=stream),
    }


NAMES = ["quantize_act", "gemv", "gemv_argmax", "tile_device", "gemv_parts", "gemv_glu", "gemv_residual_norm", "kv_slots",
         "rope_append", "attn_decode", "attn_prefill"]


@pytest.mark.parametrize("handle", ["stream", "number"])
@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_another_stream_owns_what_it_allocates(q8, name, handle):
    import torch
    call = calls(q8, torch)[name]
    want = [t.clone() for t in tensors(call(None))]
    side = torch.cuda.Stream()
    for _ in range(2):
        scratch = [torch.empty(q8.lib().q8_attn_workspace_bytes(), dtype=torch.uint8, device="cuda")]
        leave_work(torch, want + (scratch if name.startswith("attn") else []))
        got = tensors(call(side if handle == "stream" else side.cuda_stream))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert q8.device_fault() == 0


def test_the_current_stream_by_name(q8):
    """stream= naming the current stream, the default one among them, is as if it were not given."""
    import torch
    call = calls(q8, torch)["attn_decode"]
    want = call(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(call(torch.cuda.current_stream()), want)
    with torch.cuda.stream(side):
        mine = call(side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        default = call(torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(mine, want) and torch.equal(default, want)
