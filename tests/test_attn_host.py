"""The key-value cache's operators on the CPU: refusals before anything touches CUDA, the rotation table, and the
binding's checks (no compute call runs here)."""
import ctypes

import numpy as np
import pytest

import q8_block_quantized_gemv_gb300 as q8
from q8_block_quantized_gemv_gb300 import build as q8build

OK, ARG, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    q8build.build()
    return q8.lib()


def _kv(**kw):
    a = dict(k=1 << 32, v=1 << 33, k_scale=None, v_scale=None, page_stride=4 * 16 * 128, pages=10, heads=4,
             page_size=16, dim=128)
    a.update(kw)
    return q8._KV(*[a[n] for n, _ in q8._KV._fields_])


CACHES = [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(k_scale=1 << 34), ARG), (dict(v_scale=1 << 34), ARG),
    (dict(pages=0), SHAPE), (dict(heads=0), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=24), SHAPE),
    (dict(dim=96), SHAPE), (dict(dim=0), SHAPE), (dict(page_stride=4 * 16 * 128 - 128), SHAPE),
    (dict(page_stride=4 * 16 * 128 + 64), SHAPE), (dict(heads=1 << 20, page_size=1 << 12), SHAPE),
    (dict(page_stride=1 << 40), SHAPE), (dict(k=(1 << 32) + 8), ALIGN), (dict(v=(1 << 33) + 2), ALIGN),
    (dict(k_scale=(1 << 34) + 4, v_scale=1 << 35), ALIGN),
]


def _decode(lib, cache=None, **kw):
    a = dict(q=1 << 36, ldq=1024, table=1 << 37, width=8, pitch=8, lens=1 << 38, out=1 << 39, ldo=1024, R=2, heads=8,
             scale=0.1, window=0, sinks=0, work=1 << 40)
    a.update(kw)
    c = _kv() if cache is None else cache
    return lib.q8_attn_decode(a["q"], a["ldq"], ctypes.addressof(c) if c else None, a["table"], a["width"], a["pitch"],
                              a["lens"], a["out"], a["ldo"], a["R"], a["heads"], a["scale"], a["window"], a["sinks"],
                              a["work"], None)


def _prefill(lib, cache=None, **kw):
    a = dict(q=1 << 36, ldq=1024, table=1 << 37, width=8, pitch=8, lens=1 << 38, start=(1 << 38) + 64, out=1 << 39,
             ldo=1024, rows=5, R=2, heads=8, scale=0.1, window=0, sinks=0, work=1 << 40)
    a.update(kw)
    c = _kv() if cache is None else cache
    return lib.q8_attn_prefill(a["q"], a["ldq"], ctypes.addressof(c) if c else None, a["table"], a["width"],
                               a["pitch"], a["lens"], a["start"], a["out"], a["ldo"], a["rows"], a["R"], a["heads"],
                               a["scale"], a["window"], a["sinks"], a["work"], None)


def _append(lib, cache=None, **kw):
    a = dict(q=1 << 36, ldq=1024, k=1 << 37, ldk=512, v=1 << 38, ldv=512, qg=None, kg=None, eps=1e-6, table=1 << 39,
             positions=100, rot=128, pos=1 << 40, slots=1 << 41, out=1 << 42, ldo=1024, rows=3, heads=8, flags=0)
    a.update(kw)
    c = _kv() if cache is None else cache
    return lib.q8_rope_append(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["qg"], a["kg"], a["eps"],
                              a["table"], a["positions"], a["rot"], a["pos"], a["slots"], a["out"], a["ldo"],
                              ctypes.addressof(c) if c else None, a["rows"], a["heads"], a["flags"], None)


def _slots(lib, **kw):
    a = dict(cached=1 << 32, fresh=1 << 33, R=4, page=16, free=1 << 34, n_free=9, head=None, table=1 << 35, width=5,
             pitch=6, rows=7, lens=1 << 36, start=1 << 37, pos=1 << 38, slots=1 << 39, next=1 << 40)
    a.update(kw)
    return lib.q8_kv_slots(a["cached"], a["fresh"], a["R"], a["page"], a["free"], a["n_free"], a["head"], a["table"],
                           a["width"], a["pitch"], a["rows"], a["lens"], a["start"], a["pos"], a["slots"], a["next"],
                           None)


@pytest.mark.parametrize("call", [_decode, _prefill, _append])
@pytest.mark.parametrize("bad,want", CACHES)
def test_cache_refusals(lib, call, bad, want):
    assert call(lib, _kv(**bad)) == want


ATTN = [
    (dict(q=None), ARG), (dict(table=None), ARG), (dict(lens=None), ARG), (dict(out=None), ARG), (dict(work=None), ARG),
    (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG), (dict(window=-1), ARG), (dict(sinks=-1), ARG),
    (dict(out=1 << 36), ARG), (dict(out=1 << 32), ARG), (dict(work=(1 << 36) - 16), ARG), (dict(work=1 << 39), ARG),
    (dict(R=0), SHAPE), (dict(R=16385), SHAPE), (dict(heads=0), SHAPE), (dict(heads=6), SHAPE), (dict(width=0), SHAPE),
    (dict(pitch=7), SHAPE), (dict(ldq=1016), SHAPE), (dict(ldo=1016), SHAPE), (dict(width=1 << 28, pitch=1 << 28), SHAPE),
    (dict(ldq=1028), ALIGN), (dict(ldo=1028), ALIGN), (dict(q=(1 << 36) + 8), ALIGN), (dict(out=(1 << 39) + 2), ALIGN),
    (dict(work=(1 << 40) + 8), ALIGN), (dict(table=(1 << 37) + 2), ALIGN), (dict(lens=(1 << 38) + 1), ALIGN),
]


@pytest.mark.parametrize("call", [_decode, _prefill])
@pytest.mark.parametrize("bad,want", ATTN)
def test_attention_refusals(lib, call, bad, want):
    assert call(lib, **bad) == want


def test_prefill_refusals(lib):
    assert _prefill(lib, start=None) == ARG
    assert _prefill(lib, rows=0) == SHAPE
    assert _prefill(lib, start=(1 << 38) + 2) == ALIGN


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(table=None), ARG), (dict(pos=None), ARG),
    (dict(slots=None), ARG), (dict(out=None), ARG), (dict(flags=2), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(out=1 << 37), ARG), (dict(out=1 << 33), ARG), (dict(k=1 << 33), ARG),
    (dict(rows=0), SHAPE), (dict(rows=65536), SHAPE), (dict(heads=0), SHAPE), (dict(rot=12), SHAPE),
    (dict(rot=136), SHAPE), (dict(rot=-8), SHAPE), (dict(positions=0), SHAPE), (dict(ldq=1020), SHAPE),
    (dict(ldk=508), SHAPE), (dict(ldv=508), SHAPE), (dict(ldo=1016), SHAPE), (dict(ldq=1026), ALIGN),
    (dict(ldo=1028), ALIGN), (dict(q=(1 << 36) + 4), ALIGN), (dict(qg=(1 << 43) + 4), ALIGN),
    (dict(table=(1 << 39) + 8), ALIGN), (dict(slots=(1 << 41) + 4), ALIGN), (dict(pos=(1 << 40) + 2), ALIGN)])
def test_append_refusals(lib, bad, want):
    assert _append(lib, **bad) == want


@pytest.mark.parametrize("bad,want", [
    (dict(cached=None), ARG), (dict(fresh=None), ARG), (dict(free=None), ARG), (dict(table=None), ARG),
    (dict(lens=None), ARG), (dict(start=None), ARG), (dict(pos=None), ARG), (dict(slots=None), ARG),
    (dict(next=None), ARG), (dict(lens=1 << 32), ARG), (dict(next=1 << 45, head=1 << 45), ARG),
    (dict(start=(1 << 36) + 8), ARG), (dict(R=0), SHAPE), (dict(R=16385), SHAPE), (dict(page=8), SHAPE),
    (dict(page=20), SHAPE), (dict(width=0), SHAPE), (dict(pitch=4), SHAPE), (dict(rows=-1), SHAPE),
    (dict(n_free=-1), SHAPE), (dict(slots=(1 << 39) + 4), ALIGN), (dict(table=(1 << 35) + 2), ALIGN)])
def test_slots_refusals(lib, bad, want):
    assert _slots(lib, **bad) == want


def test_workspace_is_a_constant(lib):
    n = lib.q8_attn_workspace_bytes()
    assert 0 < n < 1 << 30 and n % 16 == 0


def test_rope_table():
    pytest.importorskip("torch")
    t = q8.rope_table(50, 16, 100.0, device="cpu").numpy()
    assert t.shape == (50, 16) and t.dtype == np.float32
    f = 100.0 ** (-np.arange(8) / 8)
    for p in (0, 1, 49):
        assert np.allclose(t[p], np.concatenate([np.cos(p * f), np.sin(p * f)]), atol=1e-7)
    # far positions keep their angle: fp32 products would be off by 1e-2 here
    far = q8.rope_table(200001, 8, 10000.0, device="cpu").numpy()[200000]
    assert abs(far[0] - np.cos(200000.0)) < 1e-6 and abs(far[5] - np.sin(200000.0 * 0.1)) < 1e-6


def test_rope_table_scaling():
    pytest.importorskip("torch")
    plain = q8.rope_table(400, 32, 1e4, device="cpu").numpy()
    assert np.allclose(q8.rope_table(400, 32, 1e4, ("linear", 4.0), device="cpu").numpy()[40], plain[10], atol=1e-6)
    ntk = q8.rope_table(400, 32, 1e4, ("ntk", 8.0), device="cpu").numpy()
    assert np.allclose(ntk[:, 0], plain[:, 0], atol=1e-6)                      # the fastest pair keeps its turn
    assert np.allclose(ntk[320, [15, 31]], plain[40, [15, 31]], atol=1e-6)     # the slowest is stretched by 8
    part = q8.rope_table(400, 32, 1e4, ("parts", 4.0, 2048.0, 32.0, 1.0, 1.0), device="cpu").numpy()
    assert np.allclose(part[:, 0], plain[:, 0], atol=1e-6)
    assert np.allclose(part[320, [15, 31]], plain[80, [15, 31]], atol=1e-6)
    loud = q8.rope_table(400, 32, 1e4, ("parts", 4.0, 2048.0), device="cpu").numpy()
    assert np.allclose(loud, part * (0.1 * np.log(4.0) + 1.0), atol=1e-6)
    assert np.allclose(loud[0, :16], 0.1 * np.log(4.0) + 1.0)
    with pytest.raises(ValueError):
        q8.rope_table(10, 8, 1e4, ("other", 2.0), device="cpu")
    with pytest.raises(ValueError):
        q8.rope_table(10, 7, device="cpu")


def test_binding_refuses_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q8.KVCache(x, x)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        q8.kv_slots(i, i, torch.zeros((2, 2), dtype=torch.int32), i, 16, 2)


def test_binding_refuses_tensors_of_another_device(lib):
    """Every tensor of a call is held to the cache's device, or to that of ``cached``: by tensors that say where they are."""
    torch = pytest.importorskip("torch")

    class On(torch.Tensor):
        where = 0

        def get_device(self):
            return self.where

        is_cuda = True

    class Elsewhere(On):
        where = 1

    def on(shape, dtype, cls=On):
        return torch.zeros(shape, dtype=dtype).as_subclass(cls)

    b16, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    kv = (2, 2, 16, 64)
    cache = q8.KVCache(on(kv, b16), on(kv, b16))
    with pytest.raises(ValueError):
        q8.KVCache(on(kv, b16), on(kv, b16, Elsewhere))
    attn = dict(q=((3, 128), b16), table=((3, 2), i32), lens=((3,), i32), out=((3, 128), b16),
                workspace=((lib.q8_attn_workspace_bytes(),), torch.uint8))
    chunk = dict(attn, row_start=((4,), i32))
    append = dict(q=((3, 128), f32), k=((3, 128), f32), v=((3, 128), f32), positions=((3,), i32), slots=((3,), i64),
                  table=((9, 64), f32), q_gamma=((64,), f32), k_gamma=((64,), f32), out=((3, 128), b16))
    slots = dict(cached=((3,), i32), fresh=((3,), i32), table=((3, 2), i32), free_pages=((5,), i32), head=((1,), i32))
    calls = [(q8.attn_decode, attn, dict(cache=cache)), (q8.attn_prefill, chunk, dict(cache=cache)),
             (q8.rope_append, append, dict(cache=cache)), (q8.kv_slots, slots, dict(page_size=16, rows=3))]
    for call, tensors, rest in calls:
        for name in tensors:
            args = {n: on(*a, Elsewhere if n == name else On) for n, a in tensors.items()}
            with pytest.raises(ValueError, match="device|attn_workspace|contiguous"):
                call(**args, **rest)
    for name in ("lens", "row_start", "positions", "slots", "head"):
        table = on((3, 2), i32)
        out = dict(table=table, lens=on(3, i32), row_start=on(4, i32), positions=on(3, i32), slots=on(3, i64),
                   head=on(1, i32))
        out[name] = out[name].as_subclass(Elsewhere)
        with pytest.raises(ValueError):
            q8.kv_slots(on(3, i32), on(3, i32), table, on(5, i32), 16, 3, out=out)


def test_binding_keeps_long_windows_long(lib):
    """Windows and sinks beyond 32 bits reach the library as the longest it takes, not as their low 32 bits."""
    assert [q8._int32(n) for n in (0, 1, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 10 ** 30)] == \
        [0, 1] + [2 ** 31 - 1] * 5
    assert q8._int32(-1) == -1 and q8._int32(-2 ** 32) == -1  # refused there


@pytest.mark.parametrize("base,scaling", [
    (0.0, None), (-1.0, None), (float("nan"), None), (1e4, ("linear", 0.0)), (1e4, ("linear", -2.0)), (1e4, ("linear",)),
    (1e4, ("ntk", float("inf"))), (1e4, ("parts", 4.0)), (1e4, ("parts", 4.0, 0.0)), (1e4, ("parts", 4.0, 2048.0, 0.0, 1.0)),
    (1e4, ("parts", 4.0, 2048.0, 32.0, float("nan"))), (1e4, ("other", 2.0))])
def test_rope_table_refusals(base, scaling):
    """What would fill the table with NaN, or is not there."""
    pytest.importorskip("torch")
    with pytest.raises(ValueError):
        q8.rope_table(10, 8, base, scaling, device="cpu")
