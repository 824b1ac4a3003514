"""The stated error of the 4-bit products over deep reductions whose terms all have one sign, where roundings do not cancel.

With u = 2^-24 and A = sum |x s (c - z)|: an output's carry takes K / group additions of a group's scaled sum where one warp has
all of K, each off by at most u times the carry, which is at most A.  Eight warps' and eight CTAs' carries add at most 16 u A.
Within a group the products are exact, and its at most eight MMAs of 16 rows are taken to be off by 6 u each of the group's own
sum.  So K / group + 64 units u A, and no less than 1e-5 A is promised."""
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
    yield
    assert q8.device_fault() == 0


def units(K, group):
    """The bound in units of 2^-24 sum |x s (c - z)|."""
    return max(1e-5 * 2 ** 24, K / group + 64)


def off(y, want, N):
    """The largest error in those units, where all terms are positive."""
    return ((y[:, :N].double() - want).abs() / want).max().item() * 2 ** 24


# Widths of about one wave of tiles, so that the rule on sizes has no reason to split K; depths of a few groups beside them.
SIZES = [(512, 28672, 8192, 32), (150, 28672, 19200, 32), (20, 53248, 19456, 32), (40, 65536, 19456, 64), (100, 65536, 19456, 128),
         (1, 131072, 7328, 32), (5, 65536, 7328, 32), (16, 65536, 7328, 64), (1, 32, 500, 32), (16, 128, 500, 128),
         (64, 32, 500, 32), (64, 128, 500, 128), (300, 1024, 500, 128), (300, 1024, 500, 64)]


@pytest.mark.parametrize("m,K,N,group", SIZES)
def test_equal_terms(m, K, N, group):
    """One activation a row, one code and scale a column: every group adds the same."""
    g = torch.Generator("cuda").manual_seed(K + m)
    x = (1 + torch.rand((m, 1), device="cuda", generator=g)).bfloat16()
    code = torch.randint(1, 16, (1, N), dtype=torch.uint8, device="cuda", generator=g)
    scale = (0.01 + 0.01 * torch.rand((1, N), device="cuda", generator=g)).half()
    w = q8.Weight4((code * 17).expand(K // 2, N).contiguous(), scale.expand(K // group, N).contiguous(),
                   torch.zeros((K // group, N), dtype=torch.uint8, device="cuda"))
    want = x.double() * (code.double() * scale.double()) * K
    found = off(q8.gemv4(x.expand(m, K).contiguous(), w), want, N)
    print(f"{m} x {K} x {N}, groups of {group}: {found:.1f} of {units(K, group):.1f} units ({found * 2 ** -24:.2e})")
    assert found <= units(K, group)


@pytest.mark.parametrize("m,K,N,group", SIZES)
def test_positive_terms(m, K, N, group):
    g = torch.Generator("cuda").manual_seed(K + m + 1)
    x = torch.rand((m, K), device="cuda", generator=g).bfloat16()
    codes = torch.randint(0, 256, (K // 2, N), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.rand((K // group, N), device="cuda", generator=g).half()
    w = q8.Weight4(codes, scales, torch.zeros((K // group, N), dtype=torch.uint8, device="cuda"))
    y, worst = q8.gemv4(x, w), 0.0
    for a in range(0, N, 2048):
        c = torch.stack([codes[:, a:a + 2048] & 15, codes[:, a:a + 2048] >> 4], 1).flatten(0, 1).double()
        c *= scales[:, a:a + 2048].double().repeat_interleave(group, 0)
        worst = max(worst, off(y[:, a:a + c.shape[1]], x.double() @ c, c.shape[1]))
    print(f"{m} x {K} x {N}, groups of {group}: {worst:.1f} of {units(K, group):.1f} units ({worst * 2 ** -24:.2e})")
    assert worst <= units(K, group)


@pytest.mark.parametrize("m", [1, 5, 16, 30, 100, 300])
@pytest.mark.parametrize("sizes", [(96, 1000, 33), (40, 9000, 600), (15000, 64, 8000)])
def test_bits_follow_the_widths_of_the_call(m, sizes):
    """A part's bits do not depend on what the other parts hold; alone it may be added up in another order, within the bound."""
    K, group, u = 1024, 64, 2.0 ** -24
    g = torch.Generator("cuda").manual_seed(m)

    def weight(n):
        codes = torch.randint(0, 256, (K // 2, n), dtype=torch.uint8, device="cuda", generator=g)
        return codes, (torch.randn((K // group, n), device="cuda", generator=g) * 0.01).half()

    x = torch.randn((m, K), device="cuda", generator=g).bfloat16()
    plain = [weight(n) for n in sizes]
    ws = [q8.Weight4(*w) for w in plain]
    ys = q8.gemv4_parts(x, ws)
    assert all(torch.equal(a, b) for a, b in zip(q8.gemv4_parts(x, ws), ys))
    others = [q8.Weight4(*weight(n)) for n in sizes]
    for i, n in enumerate(sizes):
        assert torch.equal(q8.gemv4_parts(x, [ws[j] if j == i else w for j, w in enumerate(others)])[i], ys[i])
        codes, scales = plain[i]
        dense = (torch.stack([codes & 15, codes >> 4], 1).flatten(0, 1).double() - 8) * scales.double().repeat_interleave(group, 0)
        want, size = x.double() @ dense, x.double().abs() @ dense.abs()
        for y in (ys[i], q8.gemv4(x, ws[i])):
            assert ((y[:, :n].double() - want).abs() <= units(K, group) * u * size).all()
