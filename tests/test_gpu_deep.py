"""The stated error of the Q8_0 products over deep reductions of equal terms, whose roundings do not cancel: the fp32 carry of an
output is rounded once a block of 32 rows, each time by at most 2^-24 of itself, where one warp has all of K; 64 units more for
the sums within a block and the joins of warps and CTAs.  Up to K = 14336 no more than 1e-5 is promised."""
import pytest
import torch

import q8_block_quantized_gemv_gb300 as q8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,K,N", [(512, 14336, 8192), (512, 28672, 8192), (150, 28672, 19200), (16, 65536, 8192), (1, 65536, 19200)])
def test_equal_terms(m, K, N):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_block_quantized_gemv_gb300 import build
    build.build()
    g = torch.Generator("cuda").manual_seed(m)
    code = torch.randint(1, 128, (1, N), dtype=torch.int8, device="cuda", generator=g)
    scale = 0.01 + 0.01 * torch.rand((1, N), device="cuda", generator=g)
    tiled = q8.tile_device(code.expand(K, N).contiguous(), scale.expand(K // 32, N).contiguous(), N)
    x = (1 + torch.rand((m, 1), device="cuda", generator=g)).bfloat16()
    y = q8.gemv(x.expand(m, K).contiguous(), *tiled, N, tiled=True)
    want = x.double() * (code.double() * scale.double()) * K
    bound = 1e-5 if K <= 14336 else (K / 32 + 64) * 2.0 ** -24
    assert ((y.double() - want).abs() <= bound * want).all()
    assert q8.device_fault() == 0
