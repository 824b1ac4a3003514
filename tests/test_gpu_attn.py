"""The paged key-value cache's operators against plain fp64 statements of their formulas: slots (equal), the append
(fp32 arithmetic, one rounding), decode and prefill attention.

Attention's tolerance, element by element, is the sum of its roundings' worst cases (u = 2^-8, bf16's unit
roundoff: 8 significant bits, values in [1, 2) 2^-7 apart):
the result's own, u |o|; the weights' rounding before they multiply v, u A with A = sum_j w_j |v_j|; over a Q8_0 cache
the rounding of a dequantized value, u A for v, and for k a score error of at most u S with S = max_j scale sum_d |q_d
k_jd|, which moves each normalised weight by at most 2 u S relatively.  fp32 sums and the exponential are covered by
2^-13 of A.  The 2-norm of the error over a whole output, where roundings average out, must stay below 4e-3 of it."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def dev():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_block_quantized_gemv_gb300 import build
    build.build()
    return torch


@pytest.fixture(scope="module")
def work(dev):
    import q8_block_quantized_gemv_gb300 as q8
    return q8.attn_workspace()


# ---- a cache with known contents ------------------------------------------------------------------------------------

class Paged:
    """Requests of given lengths over a paged cache whose unused places hold `junk`."""

    def __init__(self, torch, lens, kv_heads, dim, page, kind, seed, junk="nan", extra_width=0, pad_stride=0):
        import q8_block_quantized_gemv_gb300 as q8
        self.torch, self.lens, self.kv_heads, self.dim, self.page, self.kind = torch, lens, kv_heads, dim, page, kind
        rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n in lens]
        self.width = max(max(counts), 1) + extra_width
        pages = sum(counts) + 2
        order = rng.permutation(pages)
        self.table = np.full((len(lens), self.width), -1, dtype=np.int32)
        shape = (pages, kv_heads, page, dim)
        bad = {"nan": np.nan, "inf": np.inf, "zero": 0.0}[junk]
        self.k, self.v = [], []
        if kind == "bf16":
            raw = [np.full(shape, bad, dtype=np.float32) for _ in range(2)]
        else:
            raw = [np.full(shape, 127, dtype=np.int8) for _ in range(2)]
            scl = [np.full((*shape[:3], dim // 32), bad, dtype=np.float32) for _ in range(2)]
        at = 0
        for r, n in enumerate(lens):
            ids = order[at:at + counts[r]]
            at += counts[r]
            self.table[r, :counts[r]] = ids
            for which, keep in ((0, self.k), (1, self.v)):
                x = rng.standard_normal((n, kv_heads, dim)).astype(np.float32)
                if which == 0:
                    x[..., ::dim // 4] *= 3.0
                if kind == "bf16":
                    x = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
                    keep.append(x.astype(np.float64))
                else:
                    b = x.reshape(n, kv_heads, dim // 32, 32)
                    d = (np.abs(b).max(-1) / np.float32(127.0)).astype(np.float32)
                    q = np.clip(np.rint(b / np.maximum(d, 1e-30)[..., None]), -127, 127).astype(np.int8)
                    keep.append((q.astype(np.float64) * d[..., None].astype(np.float64)).reshape(n, kv_heads, dim))
                for i, p in enumerate(ids):
                    m = min(page, n - i * page)
                    s = slice(i * page, i * page + m)
                    if kind == "bf16":
                        raw[which][p, :, :m] = x[s].transpose(1, 0, 2)
                    else:
                        raw[which][p, :, :m] = q.reshape(n, kv_heads, dim)[s].transpose(1, 0, 2)
                        scl[which][p, :, :m] = d[s].transpose(1, 0, 2)

        def place(x, dtype, per):
            t = torch.from_numpy(x).to(dtype)
            if not pad_stride:
                return t.cuda()
            dense = int(np.prod(x.shape[1:]))
            pitch = dense + pad_stride // per
            store = torch.full((x.shape[0] * pitch,), 0, dtype=dtype, device="cuda")
            view = store.as_strided(x.shape, (pitch, *t.stride()[1:]))
            view.copy_(t)
            return view

        if kind == "bf16":
            parts = [place(x, torch.bfloat16, 1) for x in raw]
        else:
            parts = [place(x, torch.int8, 1) for x in raw] + [place(x, torch.float32, 32) for x in scl]
        self.cache = q8.KVCache(*parts)
        self.table_dev = torch.from_numpy(self.table).cuda()
        self.lens_dev = torch.tensor(lens, dtype=torch.int32, device="cuda")


def seen(pos, n, window, sinks):
    j = np.arange(n)
    ok = j <= pos
    if window:
        ok &= (pos - j < window) | (j < sinks)
    return ok


def reference(q, k, v, ok, scale):
    """One head's rows over one request: q [n, dim], k, v [len, dim], ok [n, len] -> (o, tolerance) in fp64."""
    o, t8, t16 = (np.zeros((q.shape[0], k.shape[1])) for _ in range(3))
    for i in range(q.shape[0]):
        j = np.nonzero(ok[i])[0]
        if not len(j):
            continue
        s = (k[j] @ q[i]) * scale
        big = abs(scale) * (np.abs(k[j]) @ np.abs(q[i]))
        w = np.exp(s - s.max())
        w /= w.sum()
        o[i] = w @ v[j]
        a = w @ np.abs(v[j])
        t16[i] = U * np.abs(o[i]) + (U + 2.0 ** -13) * a
        t8[i] = U * np.abs(o[i]) + (2 * U + 2 * U * big.max() + 2.0 ** -13) * a
    return o, t16, t8


def queries(torch, rows, heads, dim, seed, pad=0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((1.5 * rng.standard_normal((rows, heads * dim + pad))).astype(np.float32)).to(torch.bfloat16)
    return x.cuda(), x.float().numpy().astype(np.float64)[:, :heads * dim].reshape(rows, heads, dim)


def agree(got, want, tol):
    got = got.float().cpu().numpy().astype(np.float64).reshape(want.shape)
    assert np.all(np.isfinite(got))
    over = np.abs(got - want) - tol
    assert np.all(over <= 0), f"worst excess {over.max()} at {np.unravel_index(over.argmax(), over.shape)}"
    norm = np.linalg.norm(want)
    if norm:
        assert np.linalg.norm(got - want) <= 4e-3 * norm


def expected(p, qn, row_start, scale, window, sinks):
    """All rows' results and tolerances; row_start as prefill has it."""
    rows, heads, dim = qn.shape
    o, tol = np.zeros(qn.shape), np.zeros(qn.shape)
    group = heads // p.kv_heads
    for r, n in enumerate(p.lens):
        t0, t1 = row_start[r], row_start[r + 1]
        ok = np.stack([seen(n - (t1 - t0) + i, n, window, sinks) for i in range(t1 - t0)]) if t1 > t0 else None
        for h in range(heads):
            if t1 > t0 and n:
                a, t16, t8 = reference(qn[t0:t1, h], p.k[r][:, h // group], p.v[r][:, h // group], ok, scale)
                o[t0:t1, h], tol[t0:t1, h] = a, t16 if p.kind == "bf16" else t8
    return o, tol


# ---- decode ---------------------------------------------------------------------------------------------------------

DECODE = [
    # lens, heads, kv_heads, dim, page, window, sinks
    ([1], 1, 1, 128, 16, 0, 0),
    ([1, 2, 0, 15, 16, 17], 8, 8, 64, 16, 0, 0),
    ([63, 64, 65, 0, 129], 8, 2, 128, 48, 0, 0),
    ([300, 7], 32, 32, 128, 16, 0, 0),
    ([1000, 513], 28, 4, 64, 32, 0, 0),
    ([777], 32, 1, 128, 64, 0, 0),       # 32 query heads on one cache head
    ([500, 31], 40, 2, 64, 16, 0, 0),    # 20 on one
    ([4100], 8, 1, 128, 128, 0, 0),
    ([1000, 90, 64], 8, 2, 128, 48, 64, 0),
    ([1000, 90, 3], 8, 2, 64, 16, 1, 0),     # sees itself only
    ([1000, 90, 64], 8, 2, 128, 16, 100, 5),
    ([1000, 41], 4, 4, 64, 32, 33, 40),      # sinks reach into the window
    ([257, 10], 4, 2, 128, 16, 4000, 4),     # window longer than the request
    ([700], 4, 2, 128, 16, 20, 10000),       # every key a sink
]


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("lens,heads,kv_heads,dim,page,window,sinks", DECODE)
def test_decode(dev, work, kind, lens, heads, kv_heads, dim, page, window, sinks):
    """Every place of the cache that no row may see holds NaN (or, quantized, a NaN scale)."""
    import q8_block_quantized_gemv_gb300 as q8
    p = Paged(dev, lens, kv_heads, dim, page, kind, 11 + sum(lens))
    hide(dev, p, window, sinks)
    q, qn = queries(dev, len(lens), heads, dim, 12)
    scale = dim ** -0.5
    got = q8.attn_decode(q, p.cache, p.table_dev, p.lens_dev, window=window, sinks=sinks, workspace=work)
    agree(got, *expected(p, qn, list(range(len(lens) + 1)), scale, window, sinks))


def hide(torch, p, window, sinks):
    """NaN into the keys and values that a window hides from each request's last token."""
    if not window:
        return
    for r, n in enumerate(p.lens):
        for j in np.nonzero(~seen(n - 1, n, window, sinks))[0]:
            page, off = int(p.table[r, j // p.page]), int(j % p.page)
            if p.kind == "bf16":
                p.cache.k[page, :, off] = float("nan")
                p.cache.v[page, :, off] = float("nan")
            else:
                p.cache.k_scale[page, :, off] = float("nan")
                p.cache.v_scale[page, :, off] = float("inf")


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_decode_long_split(dev, work, kind):
    """A long context beside short ones and an idle row: parts joined over many CTAs, the same bits on every call and
    without a workspace of the caller's."""
    import q8_block_quantized_gemv_gb300 as q8
    lens = [30011, 5, 0, 2500]
    p = Paged(dev, lens, 2, 128, 64, kind, 21, junk="inf", extra_width=2)
    q, qn = queries(dev, len(lens), 8, 128, 22)
    got = q8.attn_decode(q, p.cache, p.table_dev, p.lens_dev, scale=0.1, workspace=work)
    agree(got, *expected(p, qn, list(range(5)), 0.1, 0, 0))
    for ws in (work, None):
        again = q8.attn_decode(q, p.cache, p.table_dev, p.lens_dev, scale=0.1, workspace=ws)
        assert dev.equal(got.view(dev.int16), again.view(dev.int16))


def test_decode_scores_far_apart(dev, work):
    """Scores in the thousands: the running maximum carries; one key takes all the weight."""
    import q8_block_quantized_gemv_gb300 as q8
    p = Paged(dev, [900, 333], 2, 64, 16, "bf16", 31)
    q, qn = queries(dev, 2, 4, 64, 32)
    for scale in (60.0, -60.0, 0.0):
        got = q8.attn_decode(q, p.cache, p.table_dev, p.lens_dev, scale=scale, workspace=work)
        o, tol = expected(p, qn, [0, 1, 2], scale, 0, 0)
        # fp32 scores of size |s| are off by up to dim 2^-24 |s| before the exponential
        s = abs(scale) * max(np.abs(k).max() for k in p.k) * np.abs(qn).sum(-1).max()
        tol = tol + 2 * (np.exp(64 * 2.0 ** -24 * s) - 1) * max(np.abs(v).max() for v in p.v)
        got = got.float().cpu().numpy().astype(np.float64).reshape(o.shape)
        assert np.all(np.abs(got - o) <= tol)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_decode_strides_stream_and_missing_pages(dev, work, kind):
    """Pitched q, out and table, pages apart, another stream; entries that name no page hide their tokens."""
    import q8_block_quantized_gemv_gb300 as q8
    torch = dev
    lens, page, heads, dim = [200, 130, 90], 16, 6, 128
    p = Paged(dev, lens, 2, dim, page, kind, 41, pad_stride=dim * 32)
    q, qn = queries(dev, 3, heads, dim, 42, pad=64)
    table = torch.full((3, p.width + 5), 10 ** 6, dtype=torch.int32, device="cuda")
    table[:, :p.width] = p.table_dev
    table[0, 2], table[0, 12], table[1, 0] = -1, p.cache.pages, -(2 ** 31)
    table[2, :] = -7  # nothing left to see
    out = torch.full((3, heads * dim + 32), 7.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = q8.attn_workspace()
        q8.attn_decode(q, p.cache, table[:, :p.width], p.lens_dev, q_heads=heads, out=out, workspace=ws)
    side.synchronize()
    gone = {0: list(range(32, 48)) + list(range(192, 200)), 1: list(range(16)), 2: list(range(90))}
    o, tol = np.zeros((3, heads, dim)), np.zeros((3, heads, dim))
    for r, n in enumerate(lens):
        ok = np.ones((1, n), dtype=bool)
        ok[0, gone[r]] = False
        for h in range(heads):
            a, t16, t8 = reference(qn[r:r + 1, h], p.k[r][:, h // 3], p.v[r][:, h // 3], ok, dim ** -0.5)
            o[r, h], tol[r, h] = a, t16 if kind == "bf16" else t8
    agree(out[:, :heads * dim], o, tol)
    assert torch.all(out[:, heads * dim:] == 7.0) and not np.any(out[2, :heads * dim].float().cpu().numpy())


def test_decode_length_beyond_table(dev, work):
    """lens past the table: the keys that the table has, at the position that lens says (the window counts from it)."""
    import q8_block_quantized_gemv_gb300 as q8
    p = Paged(dev, [96], 1, 64, 16, "bf16", 51)
    q, qn = queries(dev, 1, 2, 64, 52)
    lens = dev.tensor([150], dtype=dev.int32, device="cuda")
    for window, sinks in ((0, 0), (70, 3), (20, 3), (20, 0)):
        got = q8.attn_decode(q, p.cache, p.table_dev, lens, window=window, sinks=sinks, workspace=work)
        ok = seen(149, 96, window, sinks)[None]
        o, tol = np.zeros((1, 2, 64)), np.zeros((1, 2, 64))
        for h in range(2):
            o[0, h], tol[0, h], _ = reference(qn[:, h], p.k[0][:, 0], p.v[0][:, 0], ok, 64 ** -0.5)
        agree(got, o, tol)


def test_offsets_past_32_bits(dev, work):
    """Pages more than 2^31 values apart: a request over three of them, appended and attended."""
    import q8_block_quantized_gemv_gb300 as q8
    torch = dev
    stride, page, heads, dim = (1 << 31) + 4096, 16, 2, 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    views = []
    for _ in range(2):
        store = torch.empty((2 * stride + heads * page * dim,), dtype=torch.bfloat16, device="cuda")
        views.append(store.as_strided((3, heads, page, dim), (stride, page * dim, dim, 1)))
        views[-1].zero_()
    cache = q8.KVCache(*views)
    rng = np.random.default_rng(61)
    n = 41
    x = [rng.standard_normal((n, heads * dim)).astype(np.float32) for _ in range(3)]
    x = [torch.from_numpy(a).to(torch.bfloat16).float().cuda() for a in x]
    order = np.array([2, 1, 0])
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.from_numpy(order[np.arange(n) // page] * page + np.arange(n) % page).cuda()
    q = q8.rope_append(x[0], x[1], x[2], cache, pos, slots)
    table = torch.from_numpy(order.astype(np.int32)[None]).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    qn, k, v = (a.cpu().numpy().astype(np.float64).reshape(n, heads, dim) for a in x)
    o, tol = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
    ok = np.tril(np.ones((n, n), dtype=bool))
    for h in range(heads):
        o[:, h], tol[:, h], _ = reference(qn[:, h], k[:, h], v[:, h], ok, dim ** -0.5)
    agree(q8.attn_decode(q[-1:], cache, table, lens, workspace=work), o[-1:], tol[-1:])
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    agree(q8.attn_prefill(q, cache, table, lens, starts, workspace=work), o, tol)


# ---- prefill --------------------------------------------------------------------------------------------------------

PREFILL = [
    # lens, rows of each, padding rows, heads, kv_heads, dim, page, window, sinks
    ([1], [1], 0, 1, 1, 128, 16, 0, 0),
    ([5, 0, 40], [5, 0, 3], 2, 4, 2, 64, 16, 0, 0),
    ([200], [200], 0, 4, 4, 128, 16, 0, 0),
    ([131, 700, 129], [131, 1, 128], 1, 8, 2, 128, 48, 0, 0),
    ([260, 515], [257, 129], 3, 7, 1, 64, 32, 0, 0),
    ([300], [300], 0, 3, 1, 128, 64, 0, 0),
    ([700], [100], 0, 32, 1, 64, 16, 0, 0),
    ([530], [530], 0, 2, 1, 64, 16, 100, 0),
    ([530, 61], [300, 61], 0, 4, 2, 128, 48, 64, 4),
    ([530], [200], 0, 2, 2, 128, 16, 1, 0),
    ([400], [400], 0, 2, 1, 128, 16, 37, 130),
    ([900, 33, 64], [64, 33, 1], 5, 4, 4, 64, 128, 5000, 2),
    # sinks that end inside a run, at a tile's end, past a tile; a gap of one run, of none, inside the chunk
    ([700, 230], [90, 200], 0, 4, 2, 128, 16, 75, 17),
    ([800], [130], 0, 3, 1, 64, 48, 200, 128),
    ([900, 170], [140, 20], 1, 2, 1, 128, 32, 96, 129),
    ([1000], [64], 0, 4, 4, 64, 128, 33, 300),
    ([333], [100], 0, 2, 1, 64, 64, 170, 64),
    ([640], [256], 0, 4, 2, 128, 128, 129, 1),
    # many items of one tile, and of two, for each CTA: operand places are reused many steps later
    ([17] * 60, [17] * 60, 0, 32, 32, 64, 16, 0, 0),
    ([17] * 60, [17] * 60, 0, 32, 32, 128, 16, 0, 0),
    ([140] * 30, [140] * 30, 0, 48, 48, 64, 16, 0, 0),
    ([9, 33, 1, 128, 140] * 12, [9, 20, 1, 128, 140] * 12, 0, 32, 32, 64, 32, 0, 0),
]


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("lens,counts,pad,heads,kv_heads,dim,page,window,sinks", PREFILL)
def test_prefill(dev, work, kind, lens, counts, pad, heads, kv_heads, dim, page, window, sinks):
    import q8_block_quantized_gemv_gb300 as q8
    p = Paged(dev, lens, kv_heads, dim, page, kind, 71 + sum(lens))
    starts = [0, *np.cumsum(counts).tolist()]
    q, qn = queries(dev, starts[-1] + pad, heads, dim, 72)
    got = q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, dev.tensor(starts, dtype=dev.int32, device="cuda"),
                          window=window, sinks=sinks, workspace=work)
    agree(got, *expected(p, qn, starts, dim ** -0.5, window, sinks))
    assert not pad or not np.any(got[starts[-1]:].float().cpu().numpy())


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_prefill_long_context(dev, work, kind):
    """A chunk behind a long context, with padding rows in the middle of a tile: split along the cache, deterministic."""
    import q8_block_quantized_gemv_gb300 as q8
    lens, counts = [9001, 40], [150, 40]
    p = Paged(dev, lens, 2, 128, 64, kind, 81, junk="inf")
    starts = [0, 150, 190]
    q, qn = queries(dev, 200, 8, 128, 82)
    sd = dev.tensor(starts, dtype=dev.int32, device="cuda")
    got = q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, sd, workspace=work)
    agree(got, *expected(p, qn, starts, 128 ** -0.5, 0, 0))
    again = q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, sd)
    assert dev.equal(got.view(dev.int16), again.view(dev.int16))


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_prefill_nonfinite_keys_stay_with_their_rows(dev, work, kind, window, sinks):
    """Tokens of the chunk with NaN or inf keys or values: rows that do not see them are as without them; rows that do
    get what the formula gives (NaN, or inf of the value's sign where only a value is infinite)."""
    import q8_block_quantized_gemv_gb300 as q8
    torch, n, heads, dim, page = dev, 333, 4, 128, 16
    p = Paged(dev, [n], 2, dim, page, kind, 91)
    clean_q, qn = queries(dev, n, heads, dim, 92)
    bad = {100: ("k", np.nan), 171: ("v", np.inf), 230: ("v", np.nan), 300: ("v", -np.inf)}
    for j, (which, x) in bad.items():
        page_id, off = int(p.table[0, j // page]), j % page
        kv = p.k if which == "k" else p.v
        if kind == "bf16":
            getattr(p.cache, which)[page_id, :, off, 5] = float(x)
            kv[0][j, :, 5] = x
        else:
            getattr(p.cache, which + "_scale")[page_id, :, off, 0] = float(x)
            with np.errstate(invalid="ignore"):
                codes = getattr(p.cache, which)[page_id, :, off, :32].cpu().numpy().astype(np.float64)
                kv[0][j, :, :32] = codes * x
    sd = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    got = q8.attn_prefill(clean_q, p.cache, p.table_dev, p.lens_dev, sd, window=window, sinks=sinks, workspace=work)
    got = got.float().cpu().numpy().astype(np.float64).reshape(n, heads, dim)
    with np.errstate(invalid="ignore", over="ignore"):
        o, tol = expected(p, qn, [0, n], dim ** -0.5, window, sinks)
    fine = np.isfinite(o)
    assert fine[:100].all() and not fine.all()
    assert np.array_equal(np.isnan(got), np.isnan(o))
    inf = np.isinf(o)
    assert np.array_equal(got[inf], o[inf])
    assert np.all(np.abs(got[fine] - o[fine]) <= tol[fine])


def test_prefill_matches_decode(dev, work):
    """One row a request, as decode has it: within both calls' tolerance of each other."""
    import q8_block_quantized_gemv_gb300 as q8
    lens = [400, 17, 1, 0]
    p = Paged(dev, lens, 2, 128, 32, "bf16", 101)
    q, qn = queries(dev, 4, 8, 128, 102)
    a = q8.attn_decode(q, p.cache, p.table_dev, p.lens_dev, workspace=work)
    b = q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, dev.arange(5, dtype=dev.int32, device="cuda"),
                        workspace=work)
    o, tol = expected(p, qn, list(range(5)), 128 ** -0.5, 0, 0)
    agree(a, o, tol)
    agree(b, o, tol)


# ---- slots ----------------------------------------------------------------------------------------------------------

def plain_slots(cached, fresh, table, free, head, page, rows):
    table, at = table.copy(), head
    width = table.shape[1]
    pos, slots, starts = [], [], [0]
    for r, (c, f) in enumerate(zip(cached, fresh)):
        c, f = max(c, 0), max(f, 0)
        have, want = -(-c // page), min(width, -(-(c + f) // page))
        for i in range(have, want):
            table[r, i] = free[at] if 0 <= at < len(free) else -1
            at += 1
        for x in range(c, c + f):
            e = table[r, x // page] if x // page < width else -1
            pos.append(x)
            slots.append(int(e) * page + x % page if e >= 0 else -1)
        starts.append(starts[-1] + f)
    pos, slots = (pos + [-1] * rows)[:rows], (slots + [-1] * rows)[:rows]
    return table, [max(c, 0) + max(f, 0) for c, f in zip(cached, fresh)], starts, pos, slots, at


@pytest.mark.parametrize("R,page,most_cached,most_fresh,pad,short,head", [
    (1, 16, 0, 1, 0, 0, 0), (1, 16, 100, 300, 0, 0, 3), (7, 48, 200, 1, 3, 0, None), (16, 16, 500, 1, 0, 2, 0),
    (33, 32, 90, 70, -20, 0, 5), (513, 64, 300, 9, 100, 0, 0), (1200, 16, 40, 40, 1, 500, 1), (5000, 16, 33, 2, 0, 0, 0),
    (16384, 128, 4, 2, 9, 0, 0)])
def test_slots(dev, R, page, most_cached, most_fresh, pad, short, head):
    import q8_block_quantized_gemv_gb300 as q8
    torch = dev
    rng = np.random.default_rng(R + page)
    cached = rng.integers(0, most_cached + 1, R)
    fresh = rng.integers(0, most_fresh + 1, R)
    if R > 4:
        cached[1], fresh[1], fresh[2], cached[3] = -5, -2, 0, 0
    width = int(max(-(-(c + f) // page) for c, f in zip(cached, fresh))) + 1 - (2 if R == 33 else 0)
    table = np.full((R, width), -1, dtype=np.int32)
    free = rng.permutation(200000).astype(np.int32)
    at = 100000
    for r in range(R):
        for i in range(min(width, -(-max(int(cached[r]), 0) // page))):
            table[r, i] = free[at]
            at += 1
    h0 = head or 0
    need = plain_slots(cached, fresh, table, free, h0, page, 0)[-1]
    free = np.ascontiguousarray(free[:max(1, need - short)])
    rows = max(0, int(np.maximum(fresh, 0).sum()) + pad)
    dev_i = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    wide = torch.full((R, width + 3), 77, dtype=torch.int32, device="cuda")
    wide[:, :width] = torch.from_numpy(table).cuda()
    view = wide[:, :width]
    for _ in range(2):  # a second call on the table it wrote gives the same
        got = q8.kv_slots(dev_i(cached), dev_i(fresh), view, torch.from_numpy(free).cuda(), page, rows,
                          head=None if head is None else dev_i([head]))
        want = plain_slots(cached, fresh, table, free, h0, page, rows)
        for name, w in zip(("table", "lens", "row_start", "positions", "slots"), want):
            assert np.array_equal(got[name].cpu().numpy(), np.asarray(w).reshape(got[name].shape)), name
        assert got["head"].item() == want[-1]
        assert torch.all(wide[:, width:] == 77)


# ---- append ---------------------------------------------------------------------------------------------------------

def plain_append(x, gamma, eps, table, pos, rot, interleaved):
    """x [rows, heads, dim] fp64 -> (normed and rotated, the scale of its fp32 rounding)."""
    x = x.copy()
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
    mag = np.abs(x)
    if rot:
        t = table[pos][:, None, :].astype(np.float64)
        c, s = t[..., :rot // 2], t[..., rot // 2:]
        i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        a, b = x[..., i].copy(), x[..., j].copy()
        x[..., i], x[..., j] = a * c - b * s, a * s + b * c
        mag[..., i], mag[..., j] = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
    return x, mag


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("rows,heads,kv_heads,dim,page,rot,interleaved,norm", [
    (1, 1, 1, 128, 16, 128, False, "qk"), (3, 8, 2, 64, 48, 64, True, "none"), (16, 32, 32, 128, 16, 64, False, "q"),
    (37, 5, 1, 64, 16, 16, True, "k"), (130, 12, 4, 128, 32, 96, False, "qk"), (130, 12, 4, 128, 32, 104, True, "qk"),
    (9, 3, 3, 64, 16, 0, False, "none"), (9, 3, 3, 64, 16, 8, False, "qk"), (1000, 7, 7, 64, 64, 40, False, "qk"),
    # enough values for four heads a lane group, head counts that end inside one
    (601, 13, 5, 128, 16, 128, False, "qk"), (601, 13, 5, 128, 16, 72, True, "q"), (1103, 11, 7, 64, 48, 64, False, "k"),
    (1103, 11, 7, 64, 48, 24, True, "qk"), (1103, 13, 6, 64, 48, 0, False, "none")])
def test_append(dev, kind, rows, heads, kv_heads, dim, page, rot, interleaved, norm):
    import q8_block_quantized_gemv_gb300 as q8
    torch = dev
    rng = np.random.default_rng(rows + rot)
    eps, limit = 1e-5, 5000
    xs = [(2.0 * rng.standard_normal((rows, n * dim + pad))).astype(np.float32)
          for n, pad in ((heads, 32), (kv_heads, 0), (kv_heads, 4))]
    xs[0][0, :dim] = 0.0  # a head of zeros
    pages = 2 * (-(-rows // page)) + 1
    cache = q8.KVCache.empty(pages, kv_heads, page, dim, kind)
    parts = [cache.k, cache.v] + ([cache.k_scale, cache.v_scale] if kind == "q8" else [])
    for t in parts:
        t.fill_(3)
    slots = rng.permutation(pages * page)[:rows].astype(np.int64)
    pos = rng.integers(0, limit, rows).astype(np.int32)
    pos[0] = limit - 1
    if rows > 8:
        pos[2], slots[2], slots[4], slots[5] = -1, slots[2], -1, pages * page
    gq = (0.5 + rng.random(dim)).astype(np.float32) if norm in ("q", "qk") else None
    gk = (0.5 + rng.random(dim)).astype(np.float32) if norm in ("k", "qk") else None
    table = q8.rope_table(limit, rot, 10000.0) if rot else None
    tn = table.cpu().numpy() if rot else None
    d = [torch.from_numpy(x).cuda() for x in xs]
    dv = lambda g: None if g is None else torch.from_numpy(g).cuda()  # noqa: E731
    out = torch.full((rows, heads * dim + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    q8.rope_append(d[0], d[1], d[2], cache, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), table=table,
                   q_heads=heads, interleaved=interleaved, q_gamma=dv(gq), k_gamma=dv(gk), eps=eps, out=out)
    live = pos >= 0
    at = np.where(live, pos, 0)
    f64 = [x[:, :n * dim].astype(np.float64).reshape(rows, n, dim)
           for x, n in zip(xs, (heads, kv_heads, kv_heads))]
    q, qm = plain_append(f64[0], gq, eps, tn, at, rot, interleaved)
    k, km = plain_append(f64[1], gk, eps, tn, at, rot, interleaved)
    q[~live], qm[~live] = 0.0, 0.0
    # fp32: a sum of dim squares, a square root, a quotient and four products: below (dim / 4 + 16) 2^-24 of the terms
    fp = (dim / 4 + 16) * 2.0 ** -24
    got = out[:, :heads * dim].float().cpu().numpy().astype(np.float64).reshape(q.shape)
    assert np.all(np.abs(got - q) <= U * np.abs(q) + 1.01 * fp * qm + 2.0 ** -133)
    assert torch.all(out[:, heads * dim:] == 9.0)
    wrote = live & (slots >= 0) & (slots < pages * page)
    touched = np.zeros((pages, page), dtype=bool)
    for name, x, mag, rel in (("k", k, km, fp), ("v", f64[2], np.abs(f64[2]), 0.0)):
        vals = getattr(cache, name).float().cpu().numpy().astype(np.float64)
        for t in np.nonzero(wrote)[0]:
            p, o = divmod(int(slots[t]), page)
            touched[p, o] = True
            if kind == "bf16":
                assert np.all(np.abs(vals[p, :, o] - x[t]) <= U * np.abs(x[t]) + 1.01 * rel * mag[t] + 2.0 ** -133)
            else:
                sc = getattr(cache, name + "_scale")[p, :, o].cpu().numpy().astype(np.float64)
                amax = np.abs(x[t]).reshape(kv_heads, -1, 32).max(-1)
                slack = rel * mag[t].reshape(kv_heads, -1, 32).max(-1) * 1.01
                assert np.all(np.abs(sc - amax / 127) <= slack / 127 + 2.0 ** -23 * amax / 127 + 1e-45)
                err = np.abs(vals[p, :, o].reshape(kv_heads, -1, 32) * sc[..., None] - x[t].reshape(kv_heads, -1, 32))
                assert np.all(err <= (sc * 0.5001 + slack)[..., None])
    raw = [t.float().cpu().numpy() for t in parts]
    for t in raw:
        assert np.all(t.transpose(0, 2, 1, 3)[~touched] == 3)


def test_append_quantizes_as_quantize_act(dev):
    """v over a Q8_0 cache: the codes and scales of q8_quantize_act of the same (bf16-representable) values, bit for
    bit, non-finite blocks too; k's NaN position and non-finite values stay in their own head and block."""
    import q8_block_quantized_gemv_gb300 as q8
    torch, rows, heads, dim, page = dev, 20, 3, 128, 16
    x = torch.randn((rows, heads * dim), device="cuda").to(torch.bfloat16)
    x[3, 40], x[4, 200], x[5, :32] = float("inf"), float("nan"), 0.0
    x[6, 64:96] *= 1e-38
    cache = q8.KVCache.empty(2, heads, page, dim, "q8")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    pos[7] = 100  # past the table
    table = q8.rope_table(64, 32)
    q = q8.rope_append(x.float(), x.float(), x.float(), cache, pos, pos.clamp(max=31).long(), table=table)
    act = q8.quantize_act(x)
    codes, scales = act.values().view(rows, heads, dim), act.scales().view(rows, heads, dim // 32)
    for t in range(rows):
        s = min(int(pos[t]), 31)
        assert torch.equal(cache.v[s // page, :, s % page], codes[t])
        a, b = cache.v_scale[s // page, :, s % page], scales[t]
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())
    ks = cache.k_scale[31 // page, :, 31 % page]
    assert torch.all(torch.isnan(ks[:, 0])) and torch.all(torch.isfinite(ks[:, 1:]))
    turned = q.float().view(rows, heads, dim)[7]
    assert torch.all(torch.isnan(turned[:, :32])) and torch.all(torch.isfinite(turned[:, 32:]))


def test_empty_calls(dev, work):
    import q8_block_quantized_gemv_gb300 as q8
    torch = dev
    cache = q8.KVCache.empty(2, 2, 16, 64)
    none = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    i32 = torch.int32
    assert q8.attn_decode(none(0, 128), cache, none(0, 3, dt=i32), none(0, dt=i32), workspace=work).shape == (0, 128)
    got = q8.rope_append(none(0, 128, dt=torch.float32), none(0, 128, dt=torch.float32), none(0, 128, dt=torch.float32),
                         cache, none(0, dt=i32), none(0, dt=torch.int64))
    assert got.shape == (0, 128)


def test_refuses_mismatched_tensors(dev, work):
    import q8_block_quantized_gemv_gb300 as q8
    torch = dev
    cache = q8.KVCache.empty(4, 2, 16, 64)
    q = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    ok = dict(workspace=work)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(table=table.long()), dict(table=table[:1]),
                dict(lens=lens.long()), dict(lens=lens[:1]), dict(out=q.float()), dict(workspace=work[:100])):
        a = {**dict(q=q, table=table, lens=lens), **ok, **bad}
        with pytest.raises(ValueError):
            q8.attn_decode(a.pop("q"), cache, a.pop("table"), a.pop("lens"), **a)
    for kw, status in ((dict(q_heads=3), 2), (dict(scale=float("nan")), 1), (dict(window=-1), 1), (dict(sinks=-1), 1),
                       (dict(out=q), 1)):
        with pytest.raises(q8.Q8Error) as e:
            q8.attn_decode(q, cache, table, lens, **ok, **kw)
        assert e.value.status == status
    with pytest.raises(q8.Q8Error) as e:  # rows not 16-byte aligned
        q8.attn_decode(torch.zeros((2, 260), dtype=torch.bfloat16, device="cuda"), cache, table, lens, q_heads=4, **ok)
    assert e.value.status == 3


# ---- requests without rows ------------------------------------------------------------------------------------------

def scattered(torch, work, R, kind, dim, seed, every):
    """R requests, nearly all without rows (some with tokens in the cache), a short chunk every so many."""
    import q8_block_quantized_gemv_gb300 as q8
    rng = np.random.default_rng(seed)
    lens, counts = [0] * R, [0] * R
    for r in [*range(3, R, every), R - 1]:
        counts[r] = int(rng.integers(1, 40))
        lens[r] = counts[r] + int(rng.integers(0, 200))
    for r in range(5, R, 7 * every):
        if not counts[r]:
            lens[r] = 20
    p = Paged(torch, lens, 2, dim, 32, kind, seed)
    starts = [0, *np.cumsum(counts).tolist()]
    q, qn = queries(torch, starts[-1] + 2, 4, dim, seed + 1)
    sd = torch.tensor(starts, dtype=torch.int32, device="cuda")
    got = q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, sd, workspace=work)
    agree(got, *expected(p, qn, starts, dim ** -0.5, 0, 0))
    assert q8.device_fault() == 0


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_long_walks_between_items(dev, work, kind, dim):
    """Hundreds of requests without rows between two that have some: the kernel's warps walk over them one by one, at
    speeds of their own."""
    scattered(dev, work, 9000, kind, dim, 111, 250)
    scattered(dev, work, 1200, kind, dim, 112, 11)


@pytest.mark.parametrize("dim,kind,R", [
    # The list of requests is cut in shared memory: the most that have copies of their lengths beside it, and more.
    (64, "q8", 13994), (64, "q8", 13995), (64, "q8", 14336), (64, "q8", 16384), (64, "bf16", 16383), (64, "bf16", 16384),
    (128, "q8", 16384), (128, "bf16", 16384)])
def test_prefill_most_requests(dev, work, dim, kind, R):
    scattered(dev, work, R, kind, dim, R, 400)


# ---- zeros, infinities and scales far apart -------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("dim,rot,interleaved,rows", [(64, 64, False, 9), (128, 32, True, 40), (128, 0, False, 700)])
def test_append_padding_rows_are_zeros(dev, kind, dim, rot, interleaved, rows):
    """Padding rows' q are zeros whatever the norm would make of nothing: eps = 0 (0 / 0), gammas that are not finite."""
    import q8_block_quantized_gemv_gb300 as q8
    torch, heads, kv_heads, page = dev, 20, 4, 16
    rng = np.random.default_rng(dim + rows)
    xs = [rng.standard_normal((rows, n * dim)).astype(np.float32) for n in (heads, kv_heads, kv_heads)]
    pos = rng.integers(0, 100, rows).astype(np.int32)
    pos[[0, rows // 2, rows - 1]] = -1, -7, -(2 ** 31)
    gq, gk = ((0.5 + rng.random(dim)).astype(np.float32) for _ in range(2))
    table = q8.rope_table(100, rot) if rot else None
    live = pos >= 0
    for bad in (0.5, np.inf, np.nan):
        gq[dim - 1] = gk[dim - 1] = bad
        cache = q8.KVCache.empty(-(-rows // page), kv_heads, page, dim, kind)
        out = torch.full((rows, heads * dim), 9.0, dtype=torch.bfloat16, device="cuda")
        q8.rope_append(*(torch.from_numpy(x).cuda() for x in xs), cache, torch.from_numpy(pos).cuda(),
                       torch.arange(rows, device="cuda"), table=table, interleaved=interleaved,
                       q_gamma=torch.from_numpy(gq).cuda(), k_gamma=torch.from_numpy(gk).cuda(), eps=0.0, out=out)
        got = out.float().cpu().numpy().astype(np.float64).reshape(rows, heads, dim)
        assert not np.any(got[~live]) and not np.any(np.isnan(got[~live]))
        with np.errstate(invalid="ignore"):
            want, mag = plain_append(xs[0].astype(np.float64).reshape(rows, heads, dim), gq, 0.0,
                                     table.cpu().numpy() if rot else None, np.where(live, pos, 0), rot, interleaved)
        fine = np.isfinite(want) & live[:, None, None]
        fp = (dim / 4 + 16) * 2.0 ** -24
        assert np.all(np.abs(got[fine] - want[fine]) <= (U * np.abs(want) + 1.01 * fp * mag + 2.0 ** -133)[fine])


def below_all(torch, p, r, first, count):
    """Keys [first, first + count) of request r: scores of -inf from queries that are positive in the first 32 values."""
    for j in range(first, first + count):
        page, off = int(p.table[r, j // p.page]), j % p.page
        if p.kind == "bf16":
            p.cache.k[page, :, off, 0] = -float("inf")
        else:
            p.cache.k[page, :, off, :32] = -127
            p.cache.k_scale[page, :, off, 0] = float("inf")


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 128), (6, 2, 64), (20, 1, 128), (40, 2, 64)])
@pytest.mark.parametrize("first", [0, 70])
def test_decode_scores_of_minus_infinity(dev, work, kind, heads, kv_heads, dim, first):
    """Keys with a score of -inf weigh nothing, as many of them as there may be before (and after) the first finite one."""
    import q8_block_quantized_gemv_gb300 as q8
    torch, lens, page = dev, [700, 3000, 29], 16
    p = Paged(dev, lens, kv_heads, dim, page, kind, 121 + heads)
    q, qn = queries(dev, 3, heads, dim, 122)
    v = q.view(3, heads, dim)
    v[..., :32] = v[..., :32].abs() + 0.5
    qn = q.float().cpu().numpy().astype(np.float64).reshape(3, heads, dim)
    gone = {0: (first, 600), 1: (first, 2900), 2: (first if first < 29 else 0, 20)}
    for r, (at, n) in gone.items():
        below_all(torch, p, r, at, n)
    o, tol = np.zeros(qn.shape), np.zeros(qn.shape)
    for r, n in enumerate(lens):
        ok = np.ones((1, n), dtype=bool)
        ok[0, gone[r][0]:gone[r][0] + gone[r][1]] = False
        for h in range(heads):
            g = h // (heads // kv_heads)
            a, t16, t8 = reference(qn[r:r + 1, h], p.k[r][:, g], p.v[r][:, g], ok, dim ** -0.5)
            o[r, h], tol[r, h] = a, t16 if kind == "bf16" else t8
    agree(q8.attn_decode(q, p.cache, p.table_dev, p.lens_dev, workspace=work), o, tol)
    starts = torch.arange(4, dtype=torch.int32, device="cuda")
    agree(q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, starts, workspace=work), o, tol)


def value_scales(torch, p, r, factor):
    """Request r's value scales times factor [len, kv_heads, dim / 32], powers of two: in the cache and in p.v."""
    n, f = p.lens[r], torch.from_numpy(factor.astype(np.float32)).cuda()
    j = torch.arange(n, device="cuda")
    pages = p.table_dev[r].long()[j // p.page]
    p.cache.v_scale[pages, :, j % p.page] = p.cache.v_scale[pages, :, j % p.page] * f
    p.v[r] = p.v[r] * np.repeat(factor, 32, axis=2)


def far_apart(torch, lens, kv_heads, dim, page, how, seed):
    """A Q8_0 cache whose value scales lie far apart, and the keys of each request that weigh something.

    ("unseen", e): a tenth of the keys have scores some hundred below the others', weights of nothing, and value scales
    2^e times theirs; ("sink", e): one key has all the weight, and a value scale 2^-e of the others'; ("blocks", e): the
    blocks of a head in turn 2^-e, 1 and 2^e; ("all", e): every scale times 2^-e to 2^e."""
    what, e = how
    p = Paged(torch, lens, kv_heads, dim, page, "q8", seed)
    rng = np.random.default_rng(seed + 1)
    keep = []
    for r, n in enumerate(lens):
        shape = (n, kv_heads, dim // 32)
        factor, ok = np.ones(shape), np.ones(n, dtype=bool)
        if what in ("unseen", "sink"):
            if what == "unseen":
                ok[rng.permutation(n)[:n // 10]] = False
                odd, code = np.nonzero(~ok)[0], -127
                factor[~ok] = 2.0 ** e
            else:
                at = int(rng.integers(n // 2, n))
                ok[:] = False
                ok[at] = True
                odd, code = [at], 127
                factor[at] = 2.0 ** -e
            for j in odd:
                pg, off = int(p.table[r, j // page]), j % page
                p.cache.k[pg, :, off, :32] = code
                p.cache.k_scale[pg, :, off, 0] = 1.0
                p.k[r][j, :, :32] = code
        elif what == "blocks":
            factor[:] = 2.0 ** (e * (np.arange(dim // 32) % 3 - 1))
        else:
            factor = 2.0 ** rng.integers(-e, e + 1, shape)
        value_scales(torch, p, r, factor)
        keep.append(ok)
    return p, keep


FAR = [("unseen", 14), ("unseen", 20), ("unseen", 26), ("unseen", 60), ("sink", 14), ("sink", 22), ("blocks", 9),
       ("blocks", 14), ("all", 8), ("all", 13), ("all", 30)]


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (12, 1, 64)])
@pytest.mark.parametrize("how", FAR)
def test_decode_value_scales_far_apart(dev, work, how, heads, kv_heads, dim):
    """What a token's value scale is has no bearing on how well the others' values are added up."""
    import q8_block_quantized_gemv_gb300 as q8
    p, keep = far_apart(dev, [1500, 5000, 333], kv_heads, dim, 32, how, 131 + heads)
    q, _ = queries(dev, 3, heads, dim, 132)
    v = q.view(3, heads, dim)
    v[..., :32] = v[..., :32].abs() + 0.5
    qn = q.float().cpu().numpy().astype(np.float64).reshape(3, heads, dim)
    o, tol = np.zeros(qn.shape), np.zeros(qn.shape)
    for r in range(3):
        for h in range(heads):
            g = h // (heads // kv_heads)
            o[r, h], _, tol[r, h] = reference(qn[r:r + 1, h], p.k[r][:, g], p.v[r][:, g], keep[r][None], dim ** -0.5)
    agree_by_block(q8.attn_decode(q, p.cache, p.table_dev, p.lens_dev, workspace=work), o, tol)


def agree_by_block(got, want, tol):
    """agree, with the bound of the 2-norm for each block of 32 values: their sizes may be far apart."""
    agree(got, want, tol)
    diff = got.float().cpu().numpy().astype(np.float64).reshape(-1, 32) - want.reshape(-1, 32)
    # 32 roundings of u / sqrt(3) at most: their 2-norm stays below u but for one block in many millions
    assert np.all(np.linalg.norm(diff, axis=1) <= U * np.linalg.norm(want.reshape(-1, 32), axis=1))


def far_expected(p, qn, starts, keep):
    """Results, tolerances, and the 2-norms of each element's terms, w_j v_j, for causal rows.  Where a row sees keys that
    `keep` names, or the others, one kind has no weight to speak of and is left out of the sums."""
    rows, heads, dim = qn.shape
    o, tol, terms = np.zeros(qn.shape), np.zeros(qn.shape), np.zeros(qn.shape)
    group = heads // p.kv_heads
    for r, n in enumerate(p.lens):
        t0, t1 = starts[r], starts[r + 1]
        for t in range(t0, t1):
            causal = seen(n - (t1 - t0) + t - t0, n, 0, 0)
            ok = causal & keep[r] if (causal & keep[r]).any() else causal
            j = np.nonzero(ok)[0]
            for h in range(heads):
                k, v = p.k[r][:, h // group], p.v[r][:, h // group]
                o[t, h], _, tol[t, h] = (x[0] for x in reference(qn[t:t + 1, h], k, v, ok[None], dim ** -0.5))
                w = np.exp(k[j] @ qn[t, h] * dim ** -0.5 - (k[j] @ qn[t, h]).max() * dim ** -0.5)
                terms[t, h] = np.sqrt(((w / w.sum())[:, None] ** 2 * v[j] ** 2).sum(0))
    return o, tol, terms


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 128), (6, 1, 64)])
@pytest.mark.parametrize("how", FAR)
def test_prefill_value_scales_far_apart(dev, work, how, heads, kv_heads, dim):
    """The same for a chunk behind a context, a whole prompt (whose first rows see little of a tile that others see whole),
    and a few rows of a context split over many CTAs.

    Element by element as everywhere; and each block of 32 values on its own: a value is rounded twice and a weight once to
    11 bits, scores by some 2^-11 of their size: random, less than u = 2^-8 of the terms' 2-norm together, and the result
    to bf16, u of it."""
    import q8_block_quantized_gemv_gb300 as q8
    lens, counts = [700, 150, 2500], [70, 150, 5]
    p, keep = far_apart(dev, lens, kv_heads, dim, 32, how, 141 + heads)
    starts = [0, *np.cumsum(counts).tolist()]
    q, _ = queries(dev, starts[-1], heads, dim, 142)
    v = q.view(-1, heads, dim)
    v[..., :32] = v[..., :32].abs() + 0.5
    qn = q.float().cpu().numpy().astype(np.float64).reshape(-1, heads, dim)
    o, tol, terms = far_expected(p, qn, starts, keep)
    got = q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, dev.tensor(starts, dtype=dev.int32, device="cuda"),
                          workspace=work)
    agree(got, o, tol)
    off = np.linalg.norm(got.float().cpu().numpy().astype(np.float64).reshape(-1, 32) - o.reshape(-1, 32), axis=1)
    allowed = U * (np.linalg.norm(o.reshape(-1, 32), axis=1) + np.linalg.norm(terms.reshape(-1, 32), axis=1))
    assert np.all(off <= allowed), (off / allowed).max()
    assert q8.device_fault() == 0


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 4, 3), (40, 2), (1, 0)])
def test_prefill_rows_before_the_first_key(dev, work, kind, dim, window, sinks):
    """Chunks longer than their requests: rows at negative positions see nothing, the others what the window lets them,
    the widest one that the argument holds too."""
    import q8_block_quantized_gemv_gb300 as q8
    lens, counts = [10, 40, 0, 333], [20, 171, 5, 400]
    p = Paged(dev, lens, 2, dim, 16, kind, 151)
    starts = [0, *np.cumsum(counts).tolist()]
    q, qn = queries(dev, starts[-1], 6, dim, 152)
    got = q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, dev.tensor(starts, dtype=dev.int32, device="cuda"),
                          window=window, sinks=sinks, workspace=work)
    agree(got, *expected(p, qn, starts, dim ** -0.5, window, sinks))


@pytest.mark.parametrize("extra", [1, 3, 40])
def test_one_row_of_any_width(dev, work, extra):
    """A single row's column count is no pitch: any number beyond the heads' is taken, in inputs and in out."""
    import q8_block_quantized_gemv_gb300 as q8
    torch, heads, dim = dev, 4, 64
    p = Paged(torch, [77], 2, dim, 16, "bf16", 161)
    q, qn = queries(torch, 1, heads, dim, 162, pad=extra)
    want, tol = expected(p, qn, [0, 1], dim ** -0.5, 0, 0)
    starts = torch.arange(2, dtype=torch.int32, device="cuda")
    wide = lambda dt: torch.full((1, heads * dim + extra), 7.0, dtype=dt, device="cuda")  # noqa: E731
    for call in (lambda o: q8.attn_decode(q, p.cache, p.table_dev, p.lens_dev, q_heads=heads, out=o, workspace=work),
                 lambda o: q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, starts, q_heads=heads, out=o, workspace=work)):
        out = wide(torch.bfloat16)
        call(out)
        agree(out[:, :heads * dim], want, tol)
        assert torch.all(out[:, heads * dim:] == 7.0)
    x = [torch.randn((1, n * dim + extra), device="cuda") for n in (heads, 2, 2)]
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = wide(torch.bfloat16)
    q8.rope_append(*x, q8.KVCache.empty(1, 2, 16, dim), at, at.long(), q_heads=heads, out=out)
    assert torch.equal(out[:, :heads * dim], x[0][:, :heads * dim].bfloat16()) and torch.all(out[:, heads * dim:] == 7.0)


def test_windows_beyond_32_bits(dev, work):
    import q8_block_quantized_gemv_gb300 as q8
    p = Paged(dev, [90], 2, 64, 16, "bf16", 171)
    q, qn = queries(dev, 30, 4, 64, 172)
    starts = dev.tensor([0, 30], dtype=dev.int32, device="cuda")
    for window, sinks, like in ((2 ** 32 + 5, 0, (0, 0)), (2 ** 40, 3, (0, 0)), (7, 2 ** 33, (0, 0)), (7, 2 ** 31 + 1, (0, 0))):
        o, tol = expected(p, qn, [0, 30], 64 ** -0.5, *like)
        agree(q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, starts, window=window, sinks=sinks, workspace=work), o, tol)
        got = q8.attn_decode(q[-1:], p.cache, p.table_dev, p.lens_dev, window=window, sinks=sinks, workspace=work)
        agree(got, o[-1:], tol[-1:])
    with pytest.raises(q8.Q8Error):
        q8.attn_decode(q[-1:], p.cache, p.table_dev, p.lens_dev, window=-2 ** 32, workspace=work)


@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_large_values_and_rising_scores(dev, work, dim):
    """Values of 2^88 and weights that rise by 18 powers of two with every 128 keys: the sums stay finite, as the result is."""
    import q8_block_quantized_gemv_gb300 as q8
    torch, n, rows, heads, page = dev, 2000, 200, 4, 32
    p = Paged(torch, [n], 2, dim, page, "bf16", 181)
    q, _ = queries(torch, rows, heads, dim, 182)
    q.view(rows, heads, dim)[..., 0] = 1.0
    qn = q.float().cpu().numpy().astype(np.float64).reshape(rows, heads, dim)
    scale = dim ** -0.5
    pages = p.table_dev[0].long()[torch.arange(n, device="cuda") // page]
    off = torch.arange(n, device="cuda") % page
    rise = (torch.arange(n, device="cuda") / 128 * 18 * np.log(2) / scale).bfloat16()
    p.cache.k[pages, :, off, 0] = rise[:, None]
    p.cache.v[pages, :, off] *= 2.0 ** 88
    p.k[0][:, :, 0] = rise.double().cpu().numpy()[:, None]
    p.v[0] = p.v[0] * 2.0 ** 88
    o, tol = expected(p, qn, [0, rows], scale, 0, 0)
    starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    agree(q8.attn_prefill(q, p.cache, p.table_dev, p.lens_dev, starts, scale=scale, workspace=work), o, tol)
    got = q8.attn_decode(q[-1:], p.cache, p.table_dev, p.lens_dev, scale=scale, workspace=work)
    agree(got, o[-1:], tol[-1:])
