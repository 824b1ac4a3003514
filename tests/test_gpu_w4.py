"""Products over 4-bit weights on the GPU against plain 64-bit arithmetic: sizes from one row and column to whole chunks,
every group, zero points, both scale types, the gated pair, the residual norm, and the ways a program calls them."""
import numpy as np
import pytest
import torch

import oracle
import q8_block_quantized_gemv_gb300 as q8

pytestmark = pytest.mark.gpu

TOL = 1e-5  # of sum |x s (c - z)|, as stated with q8_gemv4_parts
BF16 = 2.0 ** -8  # a rounding to bf16, relative


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_block_quantized_gemv_gb300 import build
    build.build()
    yield
    assert q8.device_fault() == 0


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def plain_weight(K, N, group, zeros=False, bf16=False, seed=1):
    g = gen(seed)
    codes = torch.randint(0, 256, (K // 2, N), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.randn((K // group, N), device="cuda", generator=g) * 0.01).to(torch.bfloat16 if bf16 else torch.float16)
    z = torch.randint(0, 16, (K // group, N), dtype=torch.uint8, device="cuda", generator=g) if zeros else None
    return codes, scales, z


def dense(codes, scales, zeros=None):
    c = torch.stack([codes & 15, codes >> 4], 1).flatten(0, 1).double()
    group = c.shape[0] // scales.shape[0]
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, 0)
    return (c - z) * scales.double().repeat_interleave(group, 0)


def rows(m, K, seed=2):
    x = torch.randn((m, K), device="cuda", generator=gen(seed))
    x[:, ::37] *= 30.0
    return x.to(torch.bfloat16)


def product(x, W):
    """(x W, sum |x W|) in 64 bits."""
    return x.double() @ W, x.double().abs() @ W.abs()


def check(y, x, W, what=""):
    N = W.shape[1]
    want, size = product(x, W)
    assert y.dtype == torch.float32 and y.shape == (x.shape[0], q8.padded_n(N))
    off = (y[:, :N].double() - want).abs() - TOL * size
    assert not torch.isnan(y).any() and off.max().item() <= 0, f"{what}: off by {off.max().item()} more than allowed"
    assert not y[:, N:].any()


SIZES = [(1, 32, 1), (1, 4096, 4096), (2, 96, 40), (3, 1024, 100), (5, 5120, 3000), (7, 384, 129), (8, 2048, 512),
         (9, 640, 65), (15, 896, 257), (16, 4096, 1024), (16, 14336, 96), (17, 256, 33), (31, 1152, 300), (33, 2048, 1000),
         (64, 4096, 500), (65, 512, 127), (100, 1280, 2048), (128, 1024, 640), (129, 768, 129), (200, 4096, 96),
         (256, 512, 4096), (257, 384, 31), (300, 896, 700), (511, 640, 255), (512, 2048, 1025)]


@pytest.mark.parametrize("group,zeros,bf16", [(32, False, False), (32, True, True), (64, True, False), (64, False, True),
                                              (128, False, False), (128, True, False)])
@pytest.mark.parametrize("m,K,N", SIZES)
def test_product(m, K, N, group, zeros, bf16):
    K = -(-K // group) * group
    w = plain_weight(K, N, group, zeros, bf16, seed=m + K + N)
    x = rows(m, K, seed=m * K)
    check(q8.gemv4(x, q8.Weight4(*w)), x, dense(*w))


@pytest.mark.parametrize("m", [1, 2, 4, 8, 16, 32, 48, 96, 160, 384, 512])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_whole_numbers_are_exact(m, group):
    """Small whole activations, scales of powers of two: every sum is exact, so the product is."""
    K, N = 1024, 416
    codes, _, zeros = plain_weight(K, N, group, True, seed=m)
    scales = torch.exp2(torch.randint(-3, 4, (K // group, N), device="cuda", generator=gen(m + 1)).float()).half()
    x = torch.randint(-8, 9, (m, K), device="cuda", generator=gen(m + 2)).to(torch.bfloat16)
    want, _ = product(x, dense(codes, scales, zeros))
    y = q8.gemv4(x, q8.Weight4(codes, scales, zeros))
    assert torch.equal(y[:, :N].double(), want)


@pytest.mark.parametrize("m", [1, 6, 16, 40, 140])
def test_zero_points_up_to_127(m):
    K, N, group = 512, 96, 128
    codes, scales, _ = plain_weight(K, N, group, seed=4)
    zeros = torch.randint(0, 128, (K // group, N), dtype=torch.uint8, device="cuda", generator=gen(5))
    x = rows(m, K)
    check(q8.gemv4(x, q8.Weight4(codes, scales, zeros)), x, dense(codes, scales, zeros))


@pytest.mark.parametrize("m", [1, 7, 13, 30, 200])
def test_wide_ranges_and_values_that_are_not_finite(m):
    """Activations from 2^-120 to 2^100 keep their places; infinities and NaN stay in their row, and in their columns."""
    K, N, group = 768, 161, 64
    codes, scales, zeros = plain_weight(K, N, group, True, seed=6)
    scales = scales.float().abs().clamp(min=1e-3).half()
    x = torch.randn((m, K), device="cuda", generator=gen(7))
    x *= torch.exp2(torch.linspace(-120, 100, m, device="cuda"))[:, None]
    x = x.to(torch.bfloat16)
    check(q8.gemv4(x, q8.Weight4(codes, scales, zeros)), x, dense(codes, scales, zeros))
    x[m // 2, 5] = float("nan")
    y = q8.gemv4(x, q8.Weight4(codes, scales, zeros))
    assert torch.isnan(y[m // 2, :N]).all() and not y[:, N:].any()
    keep = torch.arange(m, device="cuda") != m // 2
    assert torch.isfinite(y[keep]).all()
    scales[3, 11] = float("inf")
    x[m // 2, 5] = 1.0
    y = q8.gemv4(x, q8.Weight4(codes, scales, zeros))
    assert torch.isfinite(y[:, :11]).all() and torch.isfinite(y[:, 12:]).all() and not torch.isfinite(y[:, 11]).any()


@pytest.mark.parametrize("m", [1, 3, 12, 25, 130, 512])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
def test_parts(m, group, zeros):
    K = 1152
    ws = [plain_weight(K, n, group, zeros, seed=n) for n in (512, 40, 33, 1)]
    x = rows(m, K)
    ys = q8.gemv4_parts(x, [q8.Weight4(*w) for w in ws])
    for y, w in zip(ys, ws):
        check(y, x, dense(*w))


def silu_bound(g, ag, u, au):
    """The products' bounds carried through silu(g) * u (|silu'| <= 1.1), and a few fp32 roundings of the result."""
    s = g * torch.sigmoid(g)
    return s * u, TOL * (1.1 * ag * u.abs() + s.abs() * au) + 1.1 * TOL ** 2 * ag * au + 1e-6 * (s * u).abs()


@pytest.mark.parametrize("m,K,N", [(1, 4096, 1000), (4, 1024, 33), (8, 512, 64), (11, 2048, 257), (16, 640, 96),
                                   (24, 1024, 160), (70, 768, 130), (128, 384, 256), (301, 1280, 300), (512, 256, 95)])
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, True)])
def test_gated_pair(m, K, N, group, zeros):
    K = -(-K // group) * group
    wg, wu = plain_weight(K, N, group, zeros, seed=8), plain_weight(K, N, group, zeros, seed=9)
    x = rows(m, K)
    out, bf = q8.gemv4_glu(x, q8.Weight4(*wg), q8.Weight4(*wu), want=("f32", "bf16"))
    want, bound = silu_bound(*product(x, dense(*wg)), *product(x, dense(*wu)))
    assert ((out[:, :N].double() - want).abs() - bound).max().item() <= 0
    assert torch.equal(out.bfloat16(), bf) and not out[:, N:].any()
    only, none = q8.gemv4_glu(x, q8.Weight4(*wg), q8.Weight4(*wu), want=("bf16",))
    assert only is None and torch.equal(none, bf)


@pytest.mark.parametrize("m,K,N", [(1, 4096, 4096), (3, 512, 33), (8, 1024, 1000), (16, 14336, 512), (40, 2048, 2048),
                                   (129, 640, 96), (512, 1024, 300)])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("place", [False, True])
def test_residual_norm(m, K, N, group, zeros, place):
    w = plain_weight(K, N, group, zeros, seed=10)
    x, Np = rows(m, K), q8.padded_n(N)
    res = torch.zeros((m, Np), device="cuda")
    res[:, :N] = torch.randn((m, N), device="cuda", generator=gen(11))
    gamma = 0.5 + torch.rand(N, device="cuda", generator=gen(12))
    y, size = product(x, dense(*w))
    want = res[:, :N].double() + y
    h, out = q8.gemv4_residual_norm(x, q8.Weight4(*w), res, gamma, 1e-6, h=res if place else None)
    tol = TOL * size + 2.0 ** -24 * want.abs()
    assert ((h[:, :N].double() - want).abs() - tol).max().item() <= 0
    assert not h[:, N:].any() and not out[:, N:].any() and (h.data_ptr() == res.data_ptr()) == place
    normed = want / (want.square().mean(1, keepdim=True) + 1e-6).sqrt() * gamma.double()

    def wide(t, fill=0.0):  # the oracle's rows are whole tiles
        full = np.full((*t.shape[:-1], Np), fill)
        full[..., :N] = t.cpu().numpy()
        return full

    bound = oracle.rmsnorm_bound(wide(want), wide(normed), wide(tol), wide(gamma).astype(np.float32), 1e-6, N)
    assert np.all(np.abs(wide(out[:, :N].double()) - wide(normed)) <= bound)


# Sizes whose tiles are one and a half waves or so: of more than 16 rows the last tiles then go apart, split over K.

@pytest.mark.parametrize("m,group,sizes", [(512, 32, (14336,)), (300, 128, (4000, 5000, 3100)), (400, 64, (128, 11800, 33, 40)),
                                           (140, 64, (21000,))])
def test_parts_of_more_than_a_wave(m, group, sizes):
    K = 640
    ws = [plain_weight(K, n, group, group == 64, seed=n) for n in sizes]
    x = rows(m, K)
    for y, w in zip(q8.gemv4_parts(x, [q8.Weight4(*w) for w in ws]), ws):
        check(y, x, dense(*w))


@pytest.mark.parametrize("m,N", [(300, 8000), (129, 12001)])
def test_gated_pair_of_more_than_a_wave(m, N):
    K = 640
    wg, wu = plain_weight(K, N, 64, True, seed=41), plain_weight(K, N, 64, True, seed=42)
    x = rows(m, K)
    out, bf = q8.gemv4_glu(x, q8.Weight4(*wg), q8.Weight4(*wu), want=("f32", "bf16"))
    want, bound = silu_bound(*product(x, dense(*wg)), *product(x, dense(*wu)))
    assert ((out[:, :N].double() - want).abs() - bound).max().item() <= 0
    assert torch.equal(out.bfloat16(), bf) and not out[:, N:].any()


def test_residual_norm_of_more_than_a_wave():
    """In place, the sums in two launches before the norm: h is the residual and the product, the rest follows from h."""
    m, K, N = 400, 640, 12001
    w = plain_weight(K, N, 128, seed=43)
    x, gamma = rows(m, K), 0.5 + torch.rand(N, device="cuda", generator=gen(44))
    h = torch.zeros((m, q8.padded_n(N)), device="cuda")
    h[:, :N] = torch.randn((m, N), device="cuda", generator=gen(45))
    y, size = product(x, dense(*w))
    want = h[:, :N].double() + y
    _, out = q8.gemv4_residual_norm(x, q8.Weight4(*w), h, gamma, 1e-6, h=h)
    assert ((h[:, :N].double() - want).abs() - TOL * size - 2.0 ** -24 * want.abs()).max().item() <= 0
    got = h[:, :N].double()  # of these very sums: the mean's and the factors' fp32 roundings, then one to bf16
    normed = got / (got.square().mean(1, keepdim=True) + 1e-6).sqrt() * gamma.double()
    assert ((out[:, :N].double() - normed).abs() - (BF16 + 1e-5) * normed.abs()).max().item() <= 0
    assert not h[:, N:].any() and not out[:, N:].any()


@pytest.mark.parametrize("m", [1, 4, 5, 12])
@pytest.mark.parametrize("group", [32, 128])
def test_so_wide_that_a_warp_takes_two_strips(m, group):
    K = 256
    ws = [plain_weight(K, n, group, True, seed=n) for n in (30001, 1000, 29)]
    x = rows(m, K)
    for y, w in zip(q8.gemv4_parts(x, [q8.Weight4(*w) for w in ws]), ws):
        check(y, x, dense(*w))
    check(q8.gemv4(x, q8.Weight4(*ws[0])), x, dense(*ws[0]))


@pytest.mark.parametrize("m", [1, 2, 3, 4])
def test_few_rows_of_a_large_weight(m):
    """Where two strips a warp are taken for the weight's size, odd strips and a K that ends inside a chunk among them."""
    w = plain_weight(8224, 4040, 32, True, seed=46)
    x = rows(m, 8224)
    check(q8.gemv4(x, q8.Weight4(*w)), x, dense(*w))


@pytest.mark.parametrize("m", [1, 7, 16, 17, 50, 70, 100, 140, 180, 250, 512])
@pytest.mark.parametrize("group,K", [(32, 32), (32, 96), (32, 160), (32, 1056), (32, 2144), (64, 64), (64, 192), (64, 1088)])
def test_depths_that_end_inside_a_chunk(m, group, K):
    """One to three groups in the last chunk of 128 rows, with and without a split of K, beside whole numbers that must be exact."""
    w = plain_weight(K, 200, group, True, seed=K)
    x = rows(m, K)
    check(q8.gemv4(x, q8.Weight4(*w)), x, dense(*w))
    scales = torch.exp2(torch.randint(-3, 4, w[1].shape, device="cuda", generator=gen(m)).float()).half()
    x = torch.randint(-8, 9, (m, K), device="cuda", generator=gen(m + 1)).to(torch.bfloat16)
    want, _ = product(x, dense(w[0], scales, w[2]))
    assert torch.equal(q8.gemv4(x, q8.Weight4(w[0], scales, w[2]))[:, :200].double(), want)


@pytest.mark.parametrize("m,K,N,group", [(1, 1056, 60001, 32), (8, 2112, 61000, 64), (16, 4096, 60100, 128), (12, 160, 90000, 32)])
def test_many_waves_of_streams(m, K, N, group):
    w = plain_weight(K, N, group, True, seed=m)
    x = rows(m, K)
    for constant in (False, True):
        check(q8.gemv4(x, q8.Weight4(*w), constant_weights=constant), x, dense(*w))


@pytest.mark.parametrize("m", [1, 16, 77, 300])
def test_same_bits_again_and_in_any_company(m):
    """A call gives the same bits again, and a row's bits do not depend on the other rows' values."""
    K, N = 2048, 600
    w = q8.Weight4(*plain_weight(K, N, 64, True, seed=13))
    x = rows(m, K)
    y = q8.gemv4(x, w)
    z = torch.randn_like(x) * 100
    z[m // 2] = x[m // 2]
    assert torch.equal(q8.gemv4(x, w), y) and torch.equal(q8.gemv4(z, w)[m // 2], y[m // 2])


@pytest.mark.parametrize("m", [1, 9, 50, 256])
def test_nothing_else_is_written(m):
    K, N = 512, 70
    w = q8.Weight4(*plain_weight(K, N, 32, seed=14))
    x = rows(m, K)
    room = torch.full((m + 2, w.Np), 7.0, device="cuda")
    q8.gemv4(x, w, y=room[1:-1])
    assert (room[0] == 7).all() and (room[-1] == 7).all()
    check(room[1:-1], x, dense(*plain_weight(K, N, 32, seed=14)))


@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("m", [1, 16, 20, 300])
def test_a_captured_layer(m, constant):
    """Products that feed each other, captured and replayed on new inputs; the weights declared constant or not."""
    K, F = 512, 768
    ws = {n: plain_weight(K, F, 128, True, seed=s) for n, s in (("gate", 15), ("up", 16))}
    ws["down"] = plain_weight(F, K, 128, True, seed=17)
    w = {n: q8.Weight4(*t) for n, t in ws.items()}
    x, res = torch.empty((m, K), dtype=torch.bfloat16, device="cuda"), torch.zeros((m, K), device="cuda")
    gamma = 0.5 + torch.rand(K, device="cuda", generator=gen(18))
    mid = torch.empty((m, F), dtype=torch.bfloat16, device="cuda")
    h, out = torch.empty((m, K), device="cuda"), torch.empty((m, K), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((m, F), device="cuda")

    def layer():
        q8.gemv4_glu(x, w["gate"], w["up"], out_bf16=mid, want=(), constant_weights=constant)
        q8.gemv4_residual_norm(mid, w["down"], res, gamma, 1e-6, h=h, out_bf16=out, constant_weights=constant)
        q8.gemv4(out, w["up"], y=y, constant_weights=constant)

    x.copy_(rows(m, K, 19))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (20, 21):
        x.copy_(rows(m, K, seed) * 0.1)
        res.copy_(torch.randn((m, K), device="cuda", generator=gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (mid, h, out, y)]
        g, ag = product(x, dense(*ws["gate"]))
        u, au = product(x, dense(*ws["up"]))
        want, bound = silu_bound(g, ag, u, au)
        assert ((got[0].double() - want).abs() - bound - BF16 * (want.abs() + bound)).max().item() <= 0
        check(got[3], got[2], dense(*ws["up"]))
        p, size = product(got[0], dense(*ws["down"]))
        want = p + res.double()
        assert ((got[1].double() - want).abs() - TOL * size - 2.0 ** -24 * want.abs()).max().item() <= 0
        layer()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (mid, h, out, y)))


def test_on_another_stream():
    K, N = 1024, 256
    ws = [plain_weight(K, N, 128, True, seed=s) for s in (22, 23)]
    side = torch.cuda.Stream()
    x, res = rows(40, K), torch.randn((40, N), device="cuda", generator=gen(24))
    gamma = torch.ones(N, device="cuda")
    torch.cuda.synchronize()
    w = [q8.Weight4(*t, stream=side) for t in ws]
    y = q8.gemv4(x, w[0], stream=side)
    ys = q8.gemv4_parts(x, w, stream=side)
    g = q8.gemv4_glu(x, *w, stream=side)[0]
    h, o = q8.gemv4_residual_norm(x, w[0], res, gamma, 1e-6, stream=side)
    side.synchronize()
    W = [dense(*t) for t in ws]
    check(y, x, W[0])
    check(ys[1], x, W[1])
    want, bound = silu_bound(*product(x, W[0]), *product(x, W[1]))
    assert ((g.double() - want).abs() - bound).max().item() <= 0
    assert torch.allclose(h, res + y, atol=0, rtol=2.0 ** -23) and torch.isfinite(o).all()


def test_two_streams_at_once():
    """Calls that overlap share nothing."""
    K, N = 4096, 2048
    w = q8.Weight4(*plain_weight(K, N, 128, seed=25))
    xs = [rows(m, K, m) for m in (1, 16, 64, 512)]
    want = [q8.gemv4(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[q8.gemv4(x, w, stream=s) for _ in range(5)] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(y, b) for y in a)


def test_host_and_device_lay_out_alike():
    for K, N, group, zeros in ((128, 33, 32, True), (192, 100, 64, False), (384, 31, 128, True)):
        codes, scales, z = plain_weight(K, N, group, zeros, seed=26)
        buf = q8.tile4(codes.cpu().numpy(), scales.cpu().numpy(), None if z is None else z.cpu().numpy())
        w = q8.Weight4(codes, scales, z)
        assert np.array_equal(w.buf.cpu().numpy(), buf)
        x = rows(3, K)
        again = q8.Weight4.of_tiled(torch.from_numpy(buf).cuda(), K, N, group, zeros)
        assert torch.equal(q8.gemv4(x, again), q8.gemv4(x, w))


def test_checkpoint_blocks():
    K, N = 256, 50
    g = np.random.default_rng(27)
    blocks = g.integers(0, 256, (N, K // 32, 18), dtype=np.uint8)
    blocks[..., :2] = (g.standard_normal((N, K // 32)) * 0.1).astype("<f2").view(np.uint8).reshape(N, K // 32, 2)
    codes, scales = q8.repack4(blocks, K, N)
    w = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    low, high = (blocks[..., 2:] & 15).astype(np.float64) - 8, (blocks[..., 2:] >> 4).astype(np.float64) - 8
    d = blocks[..., :2].copy().view("<f2").astype(np.float64)
    W = torch.from_numpy((np.concatenate([low, high], -1) * d).reshape(N, K).T.copy()).cuda()
    assert torch.equal(W, dense(*w))
    x = rows(4, K)
    check(q8.gemv4(x, q8.Weight4(*w)), x, W)


def test_what_the_binding_refuses():
    w = q8.Weight4(*plain_weight(256, 64, 64, seed=28))
    other = q8.Weight4(*plain_weight(256, 64, 32, seed=28))
    x = rows(2, 256)
    for bad in (x.float(), x[:, :128], x[0], rows(256, 2).t(), x.cpu()):
        with pytest.raises(ValueError):
            q8.gemv4(bad, w)
    for y in (torch.empty((2, 64), device="cuda").half(), torch.empty((2, 32), device="cuda"), torch.empty((2, 64))):
        with pytest.raises(ValueError):
            q8.gemv4(x, w, y=y)
    for call in (lambda: q8.gemv4(rows(513, 256), w), lambda: q8.gemv4_parts(x, [w, other]),
                 lambda: q8.gemv4_glu(x, w, other), lambda: q8.gemv4_glu(x, w, w, want=())):
        with pytest.raises(q8.Q8Error):
            call()
    with pytest.raises(ValueError):
        q8.gemv4_parts(x, [])
    with pytest.raises(ValueError):
        q8.gemv4_residual_norm(x, w, torch.zeros((2, 32), device="cuda"), torch.ones(64, device="cuda"), 1e-6)
    codes, scales, _ = plain_weight(256, 64, 64)
    for args in ((codes, scales.float()), (codes.int(), scales), (codes, scales, scales)):
        with pytest.raises(TypeError):
            q8.Weight4(*args)
    for args in ((codes, scales[:, :32].contiguous()), (codes.t(), scales), (codes, scales[:3]), (codes[:24], scales[:1])):
        with pytest.raises(ValueError):
            q8.Weight4(*args)
