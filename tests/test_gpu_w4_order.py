"""A weight laid out and used as constant at once: what orders the product's early reads behind the layout's writes, looked at in
a captured graph (the edges of a stream's launches are the same)."""
import ctypes

import pytest
import torch

import q8_block_quantized_gemv_gb300 as q8

pytestmark = pytest.mark.gpu


class Edge(ctypes.Structure):  # CUgraphEdgeData
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte),
                ("reserved", ctypes.c_ubyte * 5)]


def captured_edges(stream, work):
    """(from, to, programmatic) of every dependency among the launches of work()."""
    cuda, vp = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p
    graph, count, handle = vp(), ctypes.c_size_t(0), vp(stream.cuda_stream)
    assert cuda.cuStreamBeginCapture_v2(handle, 2) == 0  # relaxed
    try:
        work()
    finally:
        assert cuda.cuStreamEndCapture(handle, ctypes.byref(graph)) == 0
    assert cuda.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(count)) == 0
    n = count.value
    a, b, data = (vp * n)(), (vp * n)(), (Edge * n)()
    assert cuda.cuGraphGetEdges_v2(graph, a, b, data, ctypes.byref(count)) == 0 and count.value == n
    cuda.cuGraphDestroy(graph)
    return [(x, y, d.type == 1) for x, y, d in zip(a, b, data)]


@pytest.mark.parametrize("m", [2, 40])
def test_a_constant_product_starts_behind_the_layout(m):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_block_quantized_gemv_gb300 import build
    build.build()
    K, N, group = 256, 96, 64
    g = torch.Generator("cuda").manual_seed(m)
    codes = torch.randint(0, 256, (K // 2, N), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.rand((K // group, N), device="cuda", generator=g).half()
    x = torch.randn((m, K), device="cuda", generator=g).bfloat16()
    w = q8.Weight4(codes, scales)
    y = torch.empty((m, w.Np), device="cuda")
    side = torch.cuda.Stream()
    q8.gemv4(x, w, y=y, constant_weights=True)
    torch.cuda.synchronize()

    def product():
        q8.gemv4(x, w, y=y, constant_weights=True, stream=side)

    def layout():
        st = q8.lib().q8_w4_tile_device(codes.data_ptr(), scales.data_ptr(), None, K, N, group, 0, w.buf.data_ptr(),
                                        side.cuda_stream)
        assert st == 0

    twice = captured_edges(side, lambda: (product(), product()))
    assert [p for _, _, p in twice] == [True]  # a product starts early behind another
    edges = captured_edges(side, lambda: (layout(), product()))
    starts, ends = {a for a, _, _ in edges}, {b for _, b, _ in edges}
    assert len(starts - ends) == 1 and len(ends - starts) == 1 and len(edges) == len(starts)  # a chain
    assert not all(p for _, _, p in edges)  # and does not reach back to the layout


@pytest.mark.parametrize("m", [1, 16, 40])
def test_the_same_over_q8_weights(m):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K, N = 256, 128
    g = torch.Generator("cuda").manual_seed(m)
    q = torch.randint(-127, 128, (K, N), dtype=torch.int8, device="cuda", generator=g)
    s = torch.rand((K // 32, N), device="cuda", generator=g)
    x = torch.randn((m, K), device="cuda", generator=g).bfloat16()
    qt, st = q8.tile_device(q, s, N)
    y = torch.empty((m, N), device="cuda")
    side = torch.cuda.Stream()
    q8.gemv(x, qt, st, N, y=y, tiled=True, constant_weights=True)
    torch.cuda.synchronize()

    def product():
        q8.gemv(x, qt, st, N, y=y, tiled=True, constant_weights=True, stream=side)

    def layout():
        assert q8.lib().q8_tile_device(q.data_ptr(), s.data_ptr(), K, N, qt.data_ptr(), st.data_ptr(), side.cuda_stream) == 0

    assert all(p for _, _, p in captured_edges(side, lambda: (product(), product())))
    edges = captured_edges(side, lambda: (layout(), product()))
    starts, ends = {a for a, _, _ in edges}, {b for _, b, _ in edges}
    first = (starts - ends).pop()
    assert [p for a, _, p in edges if a == first] == [False]  # nothing starts early behind the layout itself
