"""Sizes and row pitches beyond the library's 32 bits: refused by the binding, never passed as their low bits (CPU; stand-ins
for tensors too large to make)."""
import numpy as np
import pytest

import q8_block_quantized_gemv_gb300 as q8
from q8_block_quantized_gemv_gb300 import build as q8build

torch = pytest.importorskip("torch")
WRAP = 2 ** 32  # arrives as 0 where only 32 bits are taken


@pytest.fixture(scope="module", autouse=True)
def lib():
    q8build.build()


class Like:
    """What the binding looks at of a tensor on GPU 0."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, dtype, pitch=None):
        self.shape, self.dtype, self.pitch = shape, dtype, shape[-1] if pitch is None else pitch

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod([int(n) for n in self.shape], dtype=object))

    def is_contiguous(self):
        return self.pitch == self.shape[-1]

    def stride(self, i=None):
        both = (self.pitch, 1)
        return both if i is None else both[i]

    def data_ptr(self):
        return 1 << 40


def test_row_pitches_of_a_choice():
    ok = Like((2, 131072), torch.float32, 2 ** 31 - 1)
    assert q8._pitched("logits", ok, torch.float32, 2, 131072, 0) == (1 << 40, 2 ** 31 - 1)
    assert q8._pitched("logits", Like((1, 64), torch.float32, WRAP + 64), torch.float32, 1, 64, 0) == (1 << 40, 64)
    for shape, pitch in (((2, 131072), WRAP + 131072), ((2, 131072), 2 ** 31), ((1, WRAP + 100), None), ((WRAP + 1, 8), None)):
        bad = Like(shape, torch.float32, pitch)
        with pytest.raises(ValueError, match="logits"):
            q8.choose(bad)
        with pytest.raises(ValueError, match="logits"):
            q8.choose(bad, 8, out=bad)
    with pytest.raises(ValueError, match="N must"):
        q8.choose(ok, 5 - WRAP)
    with pytest.raises(ValueError, match="out"):
        q8.choose(Like((2, 64), torch.float32), out=Like((2, 64), torch.float32, WRAP + 64))


def test_row_pitches_of_the_cache():
    with pytest.raises(ValueError):
        q8._rows2("q", Like((2, 512), torch.float32, WRAP + 512), torch.float32, 512, 0)
    with pytest.raises(ValueError):
        q8._table_of(Like((2, 8), torch.int32, WRAP + 8), 2, 0)
    assert q8._rows2("q", Like((1, 512), torch.float32, WRAP + 512), torch.float32, 512, 0) == (1 << 40, 512)
    assert q8._table_of(Like((2, 8), torch.int32, 16), 2, 0) == (1 << 40, 8, 16)


@pytest.mark.parametrize("K,N", [(WRAP + 32, 32), (32, WRAP + 32), (2 ** 31, 32)])
def test_weights(K, N):
    codes, scales = Like((K // 2, N), torch.uint8), Like((K // 32, N), torch.float16)
    with pytest.raises(ValueError):
        q8.Weight4(codes, scales)
    with pytest.raises(ValueError):
        q8.Weight4.of_tiled(Like((608 * 4,), torch.uint8), K, N, 32)
    with pytest.raises(ValueError, match="2.31"):
        q8.repack4(b"", K, N)
    with pytest.raises(ValueError, match="2.31"):  # as its low bits this is K = 32, of a buffer made for less
        q8.repack4(b"", 32 - WRAP, 1)
    assert q8._w4_bytes(K, N, 32, 0) == -1 and q8._w4_bytes(32, 32, WRAP + 32, 0) == -1


def test_depths_at_the_end_of_an_int():
    """The products round K up to whole 128s."""
    lib = q8.lib()
    for K in (2 ** 31 - 32, 2 ** 31 - 64, 2 ** 31 - 96):
        assert q8._w4_bytes(K, 32, 32, 0) == -1
        w = q8._W4(1 << 33, 32, 32, 0)
        assert lib.q8_gemv4(1 << 44, q8.ctypes.addressof(w), 1 << 45, 3, K, 0, None) == 2  # SHAPE
    assert q8._w4_bytes(2 ** 31 - 128, 32, 128, 0) == (2 ** 24 - 1) * (16 * 128 + 64)
    assert q8._w4_bytes(2 ** 31 - 128, 32, 32, 0) == (2 ** 26 - 4) * (16 * 32 + 64)
