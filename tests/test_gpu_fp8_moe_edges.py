"""Edges of the 8-bit projections and the experts."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_fp8 import operands, quantized, run_quantize, same_codes
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
