"""4-bit weights and the choice of a token on the CPU: the tiled form against its description, the checkpoint repack,
refusals before anything touches CUDA, and the binding's checks (no compute call runs here)."""
import ctypes

import numpy as np
import pytest

import q8_block_quantized_gemv_gb300 as q8
from q8_block_quantized_gemv_gb300 import build as q8build

OK, ARG, SHAPE, ALIGN, NOT_Q8_0 = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    q8build.build()
    return q8.lib()


def plain(K, N, group, zeros, seed=0):
    g = np.random.default_rng(seed)
    return (g.integers(0, 256, (K // 2, N), dtype=np.uint8), g.integers(0, 1 << 16, (K // group, N), dtype=np.uint16),
            g.integers(0, 128, (K // group, N), dtype=np.uint8) if zeros else None)


def untiled(buf, K, N, group, zeros):
    """Codes [K, Nt], scales and zeros [K / group, Nt] of a tiled weight, read by the header's description of it."""
    strips, unit = (N + 31) // 32, 16 * group + 64 + (32 if zeros else 0)
    u = buf.reshape(strips, K // group, unit)
    codes = np.zeros((strips, K // group, group, 32), dtype=np.uint8)
    for b in range(group // 32):
        for t in range(4):
            for j in range(2):
                for h in range(2):
                    for i in range(8):
                        at = 256 * j + 8 * (4 * i + t) + 4 * h if group == 32 else \
                            512 * (2 * (b // 2) + j) + 16 * (4 * i + t) + 4 * (2 * (b % 2) + h)
                        word = u[:, :, at:at + 4].copy().view(np.uint32)[..., 0]
                        for p in range(4):
                            codes[:, :, 32 * b + 8 * t + 2 * p, 16 * j + 8 * h + i] = (word >> (4 * p)) & 15
                            codes[:, :, 32 * b + 8 * t + 2 * p + 1, 16 * j + 8 * h + i] = (word >> (16 + 4 * p)) & 15
    scales = u[:, :, 16 * group: 16 * group + 64].copy().view(np.uint16)
    z = u[:, :, 16 * group + 64:] if zeros else None

    def flat(x):
        return None if x is None else x.transpose(1, 0, 2).reshape(K // group, 32 * strips)

    return codes.transpose(1, 2, 0, 3).reshape(K, 32 * strips), flat(scales), flat(z)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("K,N,group", [(32, 1, 32), (96, 33, 32), (64, 32, 64), (192, 70, 64), (128, 31, 128),
                                       (384, 129, 128)])
def test_tiled_form(lib, K, N, group, zeros):
    codes, scales, z = plain(K, N, group, zeros, K + N)
    buf = q8.tile4(codes, scales, z)
    assert buf.size == lib.q8_w4_bytes(K, N, group, 1 if zeros else 0)
    c, s, zz = untiled(buf, K, N, group, zeros)
    assert np.array_equal(c[0::2, :N], codes & 15) and np.array_equal(c[1::2, :N], codes >> 4)
    assert np.array_equal(s[:, :N], scales) and not s[:, N:].any() and not c[:, N:].any()
    if zeros:
        assert np.array_equal(zz[:, :N], z) and not zz[:, N:].any()


def test_bytes(lib):
    assert lib.q8_w4_bytes(4096, 4096, 128, 0) == 128 * 32 * (2048 + 64)
    assert lib.q8_w4_bytes(4096, 128256, 128, 3) == 4008 * 32 * (2048 + 96)
    assert lib.q8_w4_bytes(14336 * 4, 1 << 20, 32, 1) == (1 << 15) * 448 * 4 * (512 + 96)  # past 32 bits
    for K, N, group, flags in ((0, 32, 32, 0), (48, 32, 32, 0), (64, 32, 128, 0), (128, 0, 128, 0), (128, 32, 16, 0),
                               (128, 32, 256, 0), (128, 32, 128, 4), (-128, 32, 128, 0), (128, 2 ** 31 - 1, 128, 0)):
        assert lib.q8_w4_bytes(K, N, group, flags) == -1


def test_repack(lib):
    K, N = 96, 5
    g = np.random.default_rng(3)
    rows = g.integers(0, 16, (N, K // 32, 32), dtype=np.uint8)
    d = g.standard_normal((N, K // 32)).astype("<f2")
    blocks = np.zeros((N, K // 32, 18), dtype=np.uint8)
    blocks[..., :2] = d.view(np.uint8).reshape(N, K // 32, 2)
    blocks[..., 2:] = rows[..., :16] | (rows[..., 16:] << 4)
    codes, scales = q8.repack4(blocks, K, N)
    want = rows.reshape(N, K).T
    assert np.array_equal(codes & 15, want[0::2]) and np.array_equal(codes >> 4, want[1::2])
    assert np.array_equal(scales, d.T)
    for bad in (0x7C00, 0xFC00, 0x7E00):
        blocks[2, 1, :2] = np.array([bad], dtype="<u2").view(np.uint8)
        with pytest.raises(q8.Q8Error) as e:
            q8.repack4(blocks, K, N)
        assert e.value.status == NOT_Q8_0
    with pytest.raises(ValueError):
        q8.repack4(blocks[:4], K, N)


# ---- refusals (pointers that are never followed) -------------------------------------------------------------------

X, W, Y, Z = 1 << 32, 1 << 33, 1 << 34, 1 << 35


def weight(**kw):
    a = dict(w=W, N=96, group=64, flags=0)
    a.update(kw)
    return q8._W4(a["w"], a["N"], a["group"], a["flags"])


BAD_WEIGHTS = [(dict(w=None), ARG), (dict(flags=4), ARG), (dict(group=48), SHAPE), (dict(group=0), SHAPE),
               (dict(N=0), SHAPE), (dict(N=2 ** 31 - 1), SHAPE), (dict(w=W + 8), ALIGN)]
BAD_CALLS = [(dict(x=None), ARG), (dict(flags=2), ARG), (dict(flags=4), ARG), (dict(m=0), SHAPE), (dict(m=513), SHAPE),
             (dict(K=0), SHAPE), (dict(K=96), SHAPE), (dict(x=X + 2), ALIGN)]


def gemv(lib, w=None, **kw):
    a = dict(x=X, y=Y, m=3, K=128, flags=0)
    a.update(kw)
    w = weight() if w is None else w
    return lib.q8_gemv4(a["x"], ctypes.addressof(w), a["y"], a["m"], a["K"], a["flags"], None)


def parts(lib, w=None, n=2, y=(Y, Z), second=None, **kw):
    a = dict(x=X, m=3, K=128, flags=0)
    a.update(kw)
    arr = (q8._W4 * 8)()
    for i in range(8):
        arr[i] = weight(w=W + (i << 24))
    if w is not None:
        arr[0] = w
    if second is not None:
        arr[1] = second
    to = (ctypes.c_void_p * 8)(*(list(y) + [None] * (8 - len(y))))
    return lib.q8_gemv4_parts(a["x"], ctypes.addressof(arr), ctypes.addressof(to), n, a["m"], a["K"], a["flags"], None)


def glu(lib, w=None, up=None, **kw):
    a = dict(x=X, out=Y, bf=Z, m=3, K=128, flags=0)
    a.update(kw)
    w, up = weight() if w is None else w, weight(w=W + (1 << 24)) if up is None else up
    return lib.q8_gemv4_glu(a["x"], ctypes.addressof(w), ctypes.addressof(up), a["out"], a["bf"], a["m"], a["K"],
                            a["flags"], None)


def norm(lib, w=None, **kw):
    a = dict(x=X, res=1 << 36, gamma=1 << 37, eps=1e-6, h=Y, out=Z, m=3, K=128, flags=0)
    a.update(kw)
    w = weight() if w is None else w
    return lib.q8_gemv4_residual_norm(a["x"], ctypes.addressof(w), a["res"], a["gamma"], a["eps"], a["h"], a["out"],
                                      a["m"], a["K"], a["flags"], None)


@pytest.mark.parametrize("call", [gemv, parts, glu, norm])
@pytest.mark.parametrize("bad,want", BAD_WEIGHTS)
def test_weight_refusals(lib, call, bad, want):
    assert call(lib, weight(**bad)) == want


@pytest.mark.parametrize("call", [gemv, parts, glu, norm])
@pytest.mark.parametrize("bad,want", BAD_CALLS)
def test_call_refusals(lib, call, bad, want):
    assert call(lib, **bad) == want


def test_output_refusals(lib):
    size = lib.q8_w4_bytes(128, 96, 64, 0)
    for y, want in ((None, ARG), (Y + 4, ALIGN), (X, ARG), (X + 3 * 128 * 2 - 16, ARG), (W + size - 16, ARG),
                    (W - 3 * 96 * 4 + 16, ARG)):
        assert gemv(lib, y=y) == want
    assert parts(lib, n=0) == SHAPE and parts(lib, n=9) == SHAPE and parts(lib, n=3) == ARG
    assert parts(lib, y=(Y, Y)) == ARG and parts(lib, y=(Y, Y + 3 * 96 * 4 - 16)) == ARG
    assert parts(lib, second=weight(group=32)) == ARG and parts(lib, second=weight(flags=1)) == ARG
    assert glu(lib, out=None, bf=None) == ARG and glu(lib, out=Y, bf=Y + 16) == ARG and glu(lib, bf=X) == ARG
    assert glu(lib, out=None, bf=Z + 8) == ALIGN and glu(lib, up=weight(N=64, w=1 << 38)) == SHAPE
    assert glu(lib, up=weight(flags=2, w=1 << 38)) == ARG and glu(lib, out=W) == ARG and glu(lib, bf=W + (1 << 24)) == ARG
    for kw, want in ((dict(res=None), ARG), (dict(gamma=None), ARG), (dict(h=None), ARG), (dict(out=None), ARG),
                     (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
                     (dict(h=Y + 4), ALIGN), (dict(out=Z + 8), ALIGN), (dict(res=(1 << 36) + 2), ALIGN),
                     (dict(gamma=(1 << 37) + 1), ALIGN), (dict(h=(1 << 36) + 16), ARG), (dict(out=1 << 36), ARG),
                     (dict(out=Y + 16), ARG), (dict(h=X), ARG), (dict(out=W), ARG), (dict(gamma=Y + 4), ARG)):
        assert norm(lib, **kw) == want, kw


def tile(lib, device, **kw):
    a = dict(codes=X, scales=Y, zeros=None, K=128, N=96, group=64, flags=0, w=W)
    a.update(kw)
    args = [a[n] for n in ("codes", "scales", "zeros", "K", "N", "group", "flags", "w")]
    return lib.q8_w4_tile_device(*args, None) if device else lib.q8_w4_tile(*args)


@pytest.mark.parametrize("device", [False, True])
@pytest.mark.parametrize("bad,want", [
    (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(w=None), ARG), (dict(zeros=Z), ARG), (dict(flags=1), ARG),
    (dict(flags=8), ARG), (dict(K=96), SHAPE), (dict(group=16), SHAPE), (dict(N=-1), SHAPE), (dict(w=X), ARG),
    (dict(w=Y + 16), ARG), (dict(flags=1, zeros=W), ARG), (dict(scales=Y + 1), ALIGN), (dict(w=W + 2), ALIGN)])
def test_tile_refusals(lib, device, bad, want):
    assert tile(lib, device, **bad) == want


def choose(lib, **kw):
    a = dict(logits=X, ldl=100, out=Y, ldo=104, idx=Z, m=4, N=100)
    rules = {k: kw.pop(k) for k in list(kw) if k not in a and k != "rules"}
    no_rules = kw.pop("rules", True) is None
    a.update(kw)
    c = q8._Choice()
    for k, v in rules.items():
        setattr(c, k, v)
    return lib.q8_choose(a["logits"], a["ldl"], None if no_rules else ctypes.addressof(c), a["out"], a["ldo"], a["idx"],
                         a["m"], a["N"], None)


P = 1 << 36


@pytest.mark.parametrize("bad,want", [
    (dict(logits=None), ARG), (dict(idx=None), ARG), (dict(m=0), SHAPE), (dict(m=65536), SHAPE), (dict(N=0), SHAPE),
    (dict(ldl=99), SHAPE), (dict(ldo=99), SHAPE), (dict(N=2 ** 31 - 1, ldl=2 ** 31 - 1, ldo=2 ** 31 - 1), SHAPE),
    (dict(logits=X + 2), ALIGN), (dict(out=Y + 1), ALIGN), (dict(idx=Z + 4), ALIGN), (dict(out=X), ARG),
    (dict(out=X + 400, ldo=100), ARG), (dict(idx=X + 8), ARG), (dict(idx=Y + 8), ARG),
    (dict(history=P, history_width=5, history_pitch=5), ARG),
    (dict(history=P, lengths=P + 4096, history_width=0, history_pitch=5), SHAPE),
    (dict(history=P, lengths=P + 4096, history_width=6, history_pitch=5), SHAPE),
    (dict(history=P, lengths=P + 4096, history_width=1 << 20, history_pitch=1 << 20), SHAPE),
    (dict(history=P + 4, lengths=P + 4096, history_width=5, history_pitch=5, history_wide=1), ALIGN),
    (dict(history=P + 2, lengths=P + 4096, history_width=5, history_pitch=5), ALIGN),
    (dict(history=Y, lengths=P + 4096, history_width=5, history_pitch=5), ARG),
    (dict(bias_ids=P, bias_width=3), ARG), (dict(bias=P, bias_width=3), ARG),
    (dict(bias_ids=P, bias=P + 4096, bias_width=0), SHAPE), (dict(bias_ids=P, bias=P + 4096, bias_width=2048), SHAPE),
    (dict(bias_ids=P, bias=Y, bias_width=3), ARG), (dict(mask=P, mask_count=0, mask_pitch=4), SHAPE),
    (dict(mask=P, mask_count=4, mask_pitch=3), SHAPE), (dict(mask=Y, mask_count=4, mask_pitch=4), ARG),
    (dict(noise=P, noise_pitch=99), SHAPE), (dict(noise=Z, noise_pitch=100), ARG), (dict(temperature=P + 2), ALIGN),
    (dict(repetition=Y), ARG), (dict(mask_rows=Z), ARG), (dict(prompts=P + 1), ALIGN)])
def test_choose_refusals(lib, bad, want):
    assert choose(lib, **bad) == want


def test_binding_checks(lib):
    torch = pytest.importorskip("torch")
    codes, scales = torch.zeros((64, 8), dtype=torch.uint8), torch.zeros((2, 8), dtype=torch.float16)
    with pytest.raises(ValueError):
        q8.Weight4(codes, scales)  # not on a GPU
    with pytest.raises(ValueError):
        q8.Weight4.of_tiled(codes, 128, 8, 64)
    with pytest.raises(ValueError):
        q8.choose(torch.zeros(2, 5))
    with pytest.raises(ValueError):
        q8.tile4(codes.numpy(), scales.numpy()[:, :4])
    with pytest.raises(ValueError):
        q8.tile4(codes.numpy(), np.zeros((3, 8), dtype=np.float16))
    with pytest.raises(q8.Q8Error):
        q8.tile4(np.zeros((24, 8), np.uint8), np.zeros((1, 8), np.float16))  # a group of 48
