"""Edges of the 8-bit projections and the experts."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_fp8 import close, operands, product, quantized, run_quantize, same_codes
from tests.test_gpu_moe import Layer

pytestmark = pytest.mark.gpu

E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


@pytest.fixture(scope="module")
def abi():
    from autoregressive_decode_step_gb300 import build
    build.build()
    from autoregressive_decode_step_gb300 import abi as A
    return A


# ---------------------------------------------------------------- digits
@pytest.mark.parametrize("w,off", [(BF16, 22), (E4M3, 19)])
@pytest.mark.parametrize("n", [1, 8, 9, 40])
def test_intermediate_digits_before_bf16(abi, n, w, off):
    """Two values of the intermediate that differ by 2^-off of their size are subtracted by the down product, in front of
    a bf16 y.  gate = 64, silu(64) = 64 in fp32, up = u = 183 (2^-7 + 2^-15), and u + 2^-off: 24 bits hold either, and 128
    times the piece of x of 2^-off is no less than 2^-10 after two sixteenths, so every step is exact and y is 64 x 2^-off.
    Four pieces of e4m3 (128 u = 176 + 120 / 16 + 56 / 256 - 16 / 4096, with 2^-19 more -15 in the place of -16) hold these
    two as well."""
    d = ff = 32
    a = Layer(n, d, ff, 1, 1, x=BF16, w=w)
    gu, dn = torch.zeros(1, 2, ff, d, device="cuda"), torch.zeros(1, d, ff, device="cuda")
    gu[0, 0, :2, 3] = 64
    gu[0, 1, :2, :2], gu[0, 1, 0, 2] = 1, 1
    dn[0, :, 0], dn[0, :, 1] = 1, -1
    a.gu, a.dn = gu.to(w), dn.to(w)
    if w == E4M3:
        a.gs, a.ds = torch.ones_like(a.gs), torch.ones_like(a.ds)
    a.x = torch.zeros(n, d, device="cuda")
    a.x[:, :4] = torch.tensor([183 * 2.0 ** -7, 183 * 2.0 ** -15, 2.0 ** -off, 1.0], device="cuda")
    a.x = a.x.to(BF16)
    y, _, _ = a.run(abi)
    assert (y == 64 * 2.0 ** -off).all()


# ---------------------------------------------------------------- workspaces
def test_product_and_experts_on_one_workspace(abi):
    """One workspace, as large as the largest answer, for both operators in turn: whole and cut tiles, pairs of SMs and
    not, few and many tokens.  The outputs are those of a workspace each."""
    products = [(1, 6144, 4096), (30, 1000, 4096), (256, 1024, 4096), (300, 500, 640), (64, 2048, 8192)]
    shapes = [(1, 2048, 768, 128, 8), (64, 512, 256, 8, 2), (7, 1000, 344, 60, 4), (33, 128, 640, 3, 3)]
    space = abi.workspace(max([abi.ds_gemm_fp8_workspace_bytes(*s) for s in products] +
                              [abi.ds_moe_layer_workspace_bytes(*s) for s in shapes]))
    layers = [Layer(*s, seed=i) for i, s in enumerate(shapes)]
    ops = [operands(*s, seed=i) for i, s in enumerate(products)]

    def multiply(i, ws):
        n, rows, _ = products[i]
        y = torch.full((n, rows), math.nan, device="cuda")
        w, wsc, x, xsc = ops[i]
        abi.ds_gemm_fp8(w, wsc, x, xsc, y, ws)
        return y

    alone = [multiply(i, abi.workspace(abi.ds_gemm_fp8_workspace_bytes(*s))) for i, s in enumerate(products)]
    layer_alone = [a.run(abi)[0] for a in layers]
    for i in range(len(products)):
        for j in range(len(shapes)):
            assert torch.equal(multiply(i, space), alone[i])
            assert torch.equal(layers[j].run(abi, ws=space)[0], layer_alone[j])
    assert abi.ds_workspace_error(space) == 0


def test_two_graphs_share_a_workspace(abi):
    """A graph of products and the experts and one of the experts and a product, on one workspace, replayed in turn
    without a wait in between."""
    products = [(30, 1000, 4096), (256, 1024, 4096), (1, 6144, 4096)]
    layers = [Layer(7, 1000, 344, 60, 4, x=BF16, seed=1), Layer(33, 128, 640, 3, 3, w=E4M3, seed=2)]
    space = abi.workspace(max([abi.ds_gemm_fp8_workspace_bytes(*s) for s in products] +
                              [abi.ds_moe_layer_workspace_bytes(a.n, a.d, a.ff, a.e, a.k) for a in layers]))
    ops = [operands(*s, seed=i) for i, s in enumerate(products)]
    ys = [torch.zeros(n, rows, device="cuda") for n, rows, _ in products]
    zs = [torch.zeros_like(a.x) for a in layers]

    def multiply(i):
        w, wsc, x, xsc = ops[i]
        abi.ds_gemm_fp8(w, wsc, x, xsc, ys[i], space)

    def layer(i):
        a = layers[i]
        abi.ds_moe_layer(a.x, a.router, a.k, a.norm, a.gu, a.gs, a.dn, a.ds, a.residual, zs[i], None, None, space)

    def first():
        multiply(0)
        layer(0)
        multiply(1)

    def second():
        layer(1)
        multiply(2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for f in (first, second):
            f()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                f()
    torch.cuda.synchronize()
    eager = [t.clone() for t in ys + zs]
    for t in ys + zs:
        t.zero_()
    for _ in range(10):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t, e) for t, e in zip(ys + zs, eager))
    for i, (n, rows, cols) in enumerate(products):
        close(ys[i], *product(*ops[i]), cols)
    assert abi.ds_workspace_error(space) == 0


# ---------------------------------------------------------------- launches that overlap
@pytest.mark.parametrize("n,rows,cols", [(1, 6144, 4096), (8, 512, 4096), (64, 28672, 1024), (128, 512, 2048),
                                         (256, 1024, 4096), (700, 300, 1000)])
def test_quantise_and_multiply_back_to_back(abi, n, rows, cols):
    """Step after step into the same codes and scales, other inputs each, nothing waited for in between: every step's
    product is that of its own inputs."""
    steps, kb = 40, -(-cols // 128)
    weights, w_scales, _, _ = operands(n, rows, cols, 2)
    g = torch.Generator(device="cuda").manual_seed(n)
    size = torch.exp(torch.randn(steps, n, 1, generator=g, device="cuda"))
    x = torch.randn(steps, n, cols, generator=g, device="cuda") * size
    ld = -(-cols // 16) * 16
    q = torch.zeros(n, ld, dtype=torch.uint8, device="cuda").view(E4M3)[:, :cols]
    xs = torch.zeros(n, kb, device="cuda")
    y = torch.empty(steps, n, rows, device="cuda")
    space = abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols))
    torch.cuda.synchronize()
    for i in range(steps):
        abi.ds_fp8_quantize(x[i], 1, q, xs)
        abi.ds_gemm_fp8(weights, w_scales, q, xs, y[i], space)
    torch.cuda.synchronize()
    for i in range(steps):
        abi.ds_fp8_quantize(x[i], 1, q, xs)
        torch.cuda.synchronize()
        alone = torch.empty(n, rows, device="cuda")
        abi.ds_gemm_fp8(weights, w_scales, q, xs, alone, space)
        torch.cuda.synchronize()
        assert torch.equal(alone, y[i])
    assert abi.ds_workspace_error(space) == 0


# ---------------------------------------------------------------- quantisation of many blocks
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,pad,q_pad", [
    (3001, 1001, 0, 0), (3001, 1001, 23, 1), (2999, 1024, 0, 0), (2999, 1024, 8, 8), (2999, 1024, 23, 7), (9729, 1000, 8, 0),
    (1500, 1001, 7, 23), (1250, 1024, 0, 0), (20000, 130, 0, 6)])
def test_quantize_many_blocks(abi, rows, cols, pad, q_pad, dtype):
    """More blocks than the grid has groups, so that each takes several at a time: ends that do not fill them, rows of
    sizes of their own, whole blocks and ragged ones, rows that start on 16 bytes and that do not.  Every code and scale."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols + pad)
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x *= torch.exp(4 * torch.randn(rows, 1, generator=g, device="cuda"))
    x = (x * torch.exp(torch.randn(cols + pad, generator=g, device="cuda"))).to(dtype)[:, :cols]
    buf = torch.full((rows, cols + q_pad), 0x55, dtype=torch.uint8, device="cuda")
    q, scales = run_quantize(abi, x, 1, buf.view(E4M3)[:, :cols])
    want, scale = quantized(x, 1)
    assert np.array_equal(scales.cpu().numpy(), scale)
    same_codes(q, want)
    assert (buf[:, cols:] == 0x55).all()


# ---------------------------------------------------------------- the product, few rows and many
@pytest.mark.parametrize("n,rows,cols", [
    (1, 300, 700), (12, 300, 700), (30, 5000, 2100), (50, 300, 700), (64, 2048, 4096),  # few rows
    (128, 77 * 256, 300),                                                               # up to 128 by very many features
    (200, 300, 700), (300, 1000, 4096), (130, 301, 300)])                               # pairs of SMs, whole tiles and cut ones
def test_product_not_a_number_in_each_kernel(abi, n, rows, cols):
    """A NaN code, a NaN scale or an infinite one reaches the outputs it is part of and no other."""
    w, ws, x, xs = operands(n, rows, cols, 5)
    kb = -(-cols // 128)
    bad_x, bad_w, bad_xs = n // 2, rows - 10, n - 1
    off = torch.zeros(n, rows, dtype=torch.bool, device="cuda")
    if n > 4:  # (a single row has nothing that stays)
        x.view(torch.uint8)[bad_x, 3] = 0x7f
        xs[bad_xs, kb - 1] = math.nan
        off[bad_x], off[bad_xs] = True, True
    w.view(torch.uint8)[bad_w, cols - 1] = 0xff
    ws[1, 2] = math.inf
    off[:, bad_w], off[:, 128:256] = True, True
    y = torch.zeros(n, rows, device="cuda")
    space = abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols))
    abi.ds_gemm_fp8(w, ws, x, xs, y, space)
    assert (~torch.isfinite(y) == off).all()
    if n > 4:
        x.view(torch.uint8)[bad_x, 3] = 0
        xs[bad_xs, kb - 1] = 1
    w.view(torch.uint8)[bad_w, cols - 1] = 0
    ws[1, 2] = 1
    want, size = product(w, ws, x, xs)
    close(y[~off], want[~off], size[~off], cols)
    abi.ds_gemm_fp8(w, ws, x, xs, y, space)  # and nothing of it is left
    close(y, want, size, cols)


@pytest.mark.parametrize("n,rows,cols,pad,dtype", [
    (256, 1024, 4096, 0, torch.float32), (256, 1024, 4096, 0, BF16), (300, 1001, 2048, 2, torch.float32),
    (200, 1001, 4096, 2, BF16), (2600, 2048, 1024, 0, BF16)])
def test_pairs_captured_and_on_two_streams(abi, n, rows, cols, pad, dtype):
    """Quantisation, the pairs' product and the launch that joins cut tiles in a graph, replayed on other inputs without a
    wait in between; two streams with a workspace each.  Rows of y that start on 16 bytes and that do not."""
    w, ws, _, _ = operands(n, rows, cols, 2)
    x = torch.randn(n, cols, device="cuda")
    q, xs = torch.empty(n, cols, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(n, cols // 128, device="cuda")
    spaces = [abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols)) for _ in range(2)]

    def output():
        return torch.zeros(n, rows + pad, dtype=dtype, device="cuda")[:, :rows]

    y = output()

    def step():
        abi.ds_fp8_quantize(x, 1, q, xs)
        abi.ds_gemm_fp8(w, ws, q, xs, y, spaces[0])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    inputs = [torch.randn(n, cols, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda") for i in range(4)]
    outs = [output() for _ in inputs]
    for v, o in zip(inputs, outs):
        x.copy_(v)
        graph.replay()
        o.copy_(y)
    torch.cuda.synchronize()
    for v, o in zip(inputs, outs):
        abi.ds_fp8_quantize(v, 1, q, xs)
        close(o, *product(w, ws, q, xs), cols)
    last = outs[-1]  # of the codes and scales that lie there now
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[output() for _ in range(12)] for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(12):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                abi.ds_gemm_fp8(w, ws, q, xs, outs[i][k], spaces[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, last) for out in outs for o in out)
    assert all(abi.ds_workspace_error(s) == 0 for s in spaces)


@pytest.mark.parametrize("n,rows,cols", [
    (1, 64, 4096), (16, 160 * 128, 4096), (1, 100 * 128, 15360), (64, 1000, 14336), (64, 80 * 256, 15360), (65, 300, 4096),
    (96, 19456, 300), (100, 19457, 300), (128, 80 * 256, 15360), (128, 40000, 1000), (300, 39 * 256, 4096),
    (256, 40 * 256, 15360), (1500, 1000, 4096), (700, 1003, 8192)])
def test_product_divisions_in_bf16(abi, n, rows, cols):
    """Every division of the tiles with bf16 outputs, rows apart and not; the gaps stay as they were."""
    w, ws, x, xs = operands(n, rows, cols, n + rows + cols)
    space = abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols))
    want = product(w, ws, x, xs)
    for pad in (0, 3, 8):
        buf = torch.full((n, rows + pad), 7.0, dtype=BF16, device="cuda")
        abi.ds_gemm_fp8(w, ws, x, xs, buf[:, :rows], space)
        assert abi.ds_workspace_error(space) == 0
        close(buf[:, :rows], *want, cols)
        assert (buf[:, rows:] == 7).all()
