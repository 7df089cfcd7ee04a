"""ds_fp8_quantize and ds_gemm_fp8 against their formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def abi():
    from autoregressive_decode_step_gb300 import build
    build.build()
    from autoregressive_decode_step_gb300 import abi as A
    return A


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ---------------------------------------------------------------- quantisation
def quantized(x, br):
    """Codes and scales by the formula, in the fp32 steps that it names, on the host."""
    x = x.float().cpu().numpy()
    rows, cols = x.shape
    rb, kb = -(-rows // br), -(-cols // 128)
    pad = np.zeros((rb * br, kb * 128), np.float32)
    pad[:rows, :cols] = x
    b = pad.reshape(rb, br, kb, 128)
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.abs(b).max((1, 3))
        top = np.where(np.isfinite(top), np.maximum(top, np.float32(2.0 ** -96)), np.float32(np.nan))
        scale = (top / np.float32(448)).astype(np.float32)
        factor = (np.float32(448) / top).astype(np.float32)
        v = (b * factor[:, None, :, None]).astype(np.float32).reshape(rb * br, kb * 128)[:rows, :cols]
    return torch.from_numpy(np.ascontiguousarray(v)).to(E4M3), scale


def run_quantize(abi, x, br, q=None):
    rows, cols = x.shape
    q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda").view(E4M3) if q is None else q
    scales = torch.empty(-(-rows // br), -(-cols // 128), device="cuda")
    abi.ds_fp8_quantize(x, br, q, scales)
    return q, scales


def same_codes(q, want):
    a, b = bits(q), bits(want)
    nan = (b & 0x7f) == 0x7f  # a NaN's sign is not part of the formula
    assert np.array_equal((a & 0x7f) == 0x7f, nan)
    assert np.array_equal(a[~nan], b[~nan])


@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 127, 0), (3, 128, 0), (2, 129, 0), (129, 130, 3), (128, 256, 8),
                                           (7, 4096, 0), (300, 1000, 24), (1025, 392, 0), (64, 14336, 0)])
def test_quantize(abi, rows, cols, pad, dtype, br):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x = (x * torch.exp(2 * torch.randn(cols + pad, generator=g, device="cuda"))).to(dtype)[:, :cols]
    q, scales = run_quantize(abi, x, br)
    want, scale = quantized(x, br)
    assert np.array_equal(scales.cpu().numpy(), scale)
    same_codes(q, want)


@pytest.mark.parametrize("br", [1, 128])
def test_quantize_extremes(abi, br):
    """Zeros, the least and largest numbers, ties, signs; NaN and infinities fill their own block and no other."""
    x = torch.zeros(256, 640, device="cuda")
    x[0, 0], x[0, 128:131] = 3e38, torch.tensor([1e-45, -2.0 ** -100, 2.0 ** -97], device="cuda")
    x[1, 256:272] = torch.arange(16, device="cuda") * (448 / 256) / 16 - 7
    x[128:, :] = 1.0
    x[130, 5], x[140, 200], x[200, 400] = math.nan, math.inf, -math.inf
    x[255, 512:] = 448 * 2.0 ** torch.arange(-127, 1, device="cuda").float()
    q, scales = run_quantize(abi, x, br)
    want, scale = quantized(x, br)
    assert np.array_equal(scales.cpu().numpy(), scale, equal_nan=True)
    same_codes(q, want)
    assert np.isnan(scale).sum() == 3


def test_quantize_views_and_gaps(abi):
    """Rows that start off 16 bytes, codes into rows of a wider buffer: the gaps stay as they were."""
    wide = torch.randn(37, 400, device="cuda").to(torch.bfloat16)
    for off, cols in ((0, 300), (1, 300), (8, 392), (3, 129)):
        x = wide[:, off:off + cols]
        buf = torch.full((37, 512), 0x55, dtype=torch.uint8, device="cuda")
        q = buf.view(E4M3)[:, off:off + cols]
        _, scales = run_quantize(abi, x, 1, q)
        want, scale = quantized(x, 1)
        assert np.array_equal(scales.cpu().numpy(), scale)
        same_codes(q, want)
        assert (buf[:, :off] == 0x55).all() and (buf[:, off + cols:] == 0x55).all()


def test_quantize_offsets_past_32_bits(abi):
    rows, cols = 70000, 32768  # 2.3e9 values
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, cols, device="cuda").to(torch.bfloat16)
    q, scales = run_quantize(abi, x, 1)
    want, scale = quantized(x[-3:], 1)
    assert np.array_equal(scales[-3:].cpu().numpy(), scale)
    same_codes(q[-3:], want)
    assert not q[:5].view(torch.uint8).any()


# ---------------------------------------------------------------- product
def operands(n, rows, cols, seed=0):
    """Codes with rows a multiple of 16 bytes apart, and scales of many sizes."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes(r):
        ld = -(-cols // 16) * 16 + 16
        return torch.randn(r, ld, generator=g, device="cuda").mul_(40).clamp_(-448, 448).to(E4M3)[:, :cols]

    kb = -(-cols // 128)
    xs = torch.exp(torch.randn(n, kb, generator=g, device="cuda"))
    ws = torch.exp(torch.randn(-(-rows // 128), kb, generator=g, device="cuda"))
    return codes(rows), ws, codes(n), xs


def product(w, ws, x, xs):
    """(result, sum of magnitudes) in 64 bits."""
    cols = w.shape[1]
    wd = w.double() * ws.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :cols]
    xd = x.double() * xs.double().repeat_interleave(128, 1)[:, :cols]
    return xd @ wd.t(), xd.abs() @ wd.abs().t()


def close(y, want, size, cols):
    """Products of codes are exact in fp32; a block's sum has up to 128 roundings or cuts, the blocks' sum one each
    and the scale's two: 2^-23 of the sum of magnitudes each.  bf16: its own half step on top."""
    bound = (128 + -(-cols // 128) + 2) * 2.0 ** -23 * size
    if y.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    assert ((y.double() - want).abs() <= bound).all()


SIZES = [(1, 1, 1), (1, 128, 128), (1, 6144, 4096), (2, 129, 127), (3, 1000, 1416), (16, 256, 512), (17, 300, 300),
         (32, 640, 4096), (33, 128, 16), (64, 4096, 1024), (100, 777, 2000), (128, 512, 640), (129, 1024, 4097),
         (200, 130, 14336), (256, 512, 2048), (257, 129, 129), (333, 1000, 1416), (1000, 5000, 256), (2049, 2304, 512)]


@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,rows,cols", SIZES)
def test_product(abi, n, rows, cols, y_dtype):
    w, ws, x, xs = operands(n, rows, cols, n + rows + cols)
    y = torch.full((n, rows), math.nan, dtype=y_dtype, device="cuda")
    space = abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols))
    abi.ds_gemm_fp8(w, ws, x, xs, y, space)
    assert abi.ds_workspace_error(space) == 0
    close(y, *product(w, ws, x, xs), cols)


def test_product_digits(abi):
    """Sums of many equal products: what a cut in every addition would lose adds up."""
    n, rows, cols = 40, 256, 8192
    w = torch.full((rows, cols), 1.75, device="cuda").to(E4M3)
    x = torch.full((n, cols), 1.625, device="cuda").to(E4M3)
    xs, ws = torch.full((n, 64), 1.0 / 3, device="cuda"), torch.full((2, 64), 0.7, device="cuda")
    y = torch.empty(n, rows, device="cuda")
    abi.ds_gemm_fp8(w, ws, x, xs, y, abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols)))
    want, _ = product(w, ws, x, xs)
    # a block's sum of 128 such products, 364, is exact: 2 roundings of the scale, 64 of the sum
    assert ((y.double() - want).abs() <= 66 * 2.0 ** -24 * want).all()


def test_product_not_a_number(abi):
    """A NaN code or scale reaches the outputs it is part of and no other."""
    n, rows, cols = 70, 300, 700
    w, ws, x, xs = operands(n, rows, cols, 5)
    x.view(torch.uint8)[7, 3] = 0x7f
    w.view(torch.uint8)[290, 699] = 0xff
    xs[9, 5], ws[1, 2] = math.nan, math.inf
    y = torch.empty(n, rows, device="cuda")
    abi.ds_gemm_fp8(w, ws, x, xs, y, abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols)))
    off = torch.zeros(n, rows, dtype=torch.bool, device="cuda")
    off[7], off[9], off[:, 290], off[:, 128:256] = True, True, True, True
    assert (~torch.isfinite(y) == off).all()
    fine = torch.where(off, 0.0, 1.0).bool()
    x.view(torch.uint8)[7, 3] = 0
    w.view(torch.uint8)[290, 699] = 0
    xs[9, 5], ws[1, 2] = 1, 1
    want, size = product(w, ws, x, xs)
    close(y[fine], want[fine], size[fine], cols)


def test_product_rows_apart_and_neighbours(abi):
    """Y in a wider buffer; one workspace for calls of several sizes, in turn."""
    space = abi.workspace(max(abi.ds_gemm_fp8_workspace_bytes(n, r, c) for n, r, c in SIZES + [(1, 153 * 128, 384)]))
    for n, rows, cols in ((256, 512, 2048), (5, 300, 1000), (300, 500, 640), (1, 6144, 4096), (2049, 2304, 512),
                          (40, 1000, 2000), (1, 153 * 128, 384), (5, 300, 1000)):
        w, ws, x, xs = operands(n, rows, cols, 3)
        buf = torch.full((n, rows + 9), 7.0, device="cuda")
        y = buf[:, 4:4 + rows]
        abi.ds_gemm_fp8(w, ws, x, xs, y, space)
        close(y, *product(w, ws, x, xs), cols)
        assert (buf[:, :4] == 7).all() and (buf[:, 4 + rows:] == 7).all()
    assert abi.ds_workspace_error(space) == 0


def test_product_is_the_same_each_time(abi):
    for n, rows, cols in ((1, 6144, 4096), (30, 1000, 4096), (256, 1024, 4096), (700, 2000, 1000)):
        w, ws, x, xs = operands(n, rows, cols, 1)
        space = abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols))
        first = None
        for _ in range(5):
            y = torch.empty(n, rows, device="cuda")
            abi.ds_gemm_fp8(w, ws, x, xs, y, space)
            first = y if first is None else first
            assert torch.equal(first, y)


def test_product_captured_and_on_two_streams(abi):
    """Quantisation and product in a graph, replayed on other inputs; two streams with a workspace each."""
    n, rows, cols = 48, 1500, 2048
    w, ws, _, _ = operands(n, rows, cols, 2)
    x = torch.randn(n, cols, device="cuda")
    q, xs = torch.empty(n, cols, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(n, cols // 128, device="cuda")
    y = torch.empty(n, rows, device="cuda")
    spaces = [abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols)) for _ in range(2)]

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
    for seed in range(3):
        x.copy_(torch.randn(n, cols, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        close(y, *product(w, ws, q, xs), cols)
        want, _ = quantized(x, 1)
        same_codes(q, want)
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            outs.append([torch.empty(n, rows, device="cuda") for _ in range(20)])
    torch.cuda.synchronize()
    for k in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                abi.ds_gemm_fp8(w, ws, q, xs, outs[i][k], spaces[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for out in outs for o in out)


def test_product_offsets_past_32_bits(abi):
    """Weights and outputs whose byte offsets pass 2^32."""
    n, rows, cols = 2, 140000, 32768
    w = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda").view(E4M3)
    ws = torch.ones(-(-rows // 128), cols // 128, device="cuda")
    _, _, x, xs = operands(n, 1, cols, 4)
    w[-200:] = operands(200, 1, cols, 6)[2]
    y = torch.empty(n, rows, device="cuda")
    abi.ds_gemm_fp8(w, ws, x, xs, y, abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols)))
    assert not y[:, :-200].any()
    close(y[:, -200:], *product(w[-200:], ws[-2:].clone().fill_(1), x, xs), cols)
    del w
    n, rows, cols = 40000, 60000, 128
    w, ws, x, xs = operands(n, rows, cols, 8)
    y = torch.empty(n, rows, dtype=torch.bfloat16, device="cuda")
    abi.ds_gemm_fp8(w, ws, x, xs, y, abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols)))
    for s in (slice(0, 64), slice(n - 64, n)):
        close(y[s], *product(w, ws, x[s], xs[s]), cols)


# Few tiles with long sums (cut in pieces in line with the tiles), many with very long ones (equal runs that pass from
# tile to tile), whole tiles in rounds before cut ones; features that are more tiles than pairs of SMs.
@pytest.mark.parametrize("n,rows,cols", [
    (1, 64, 4096), (16, 160 * 128, 4096), (1, 100 * 128, 15360), (64, 1000, 14336), (64, 80 * 256, 15360), (65, 300, 4096),
    (96, 19456, 300), (100, 19457, 300), (128, 80 * 256, 15360), (128, 40000, 1000), (300, 39 * 256, 4096),
    (256, 40 * 256, 15360), (1500, 1000, 4096)])
def test_product_divisions(abi, n, rows, cols):
    w, ws, x, xs = operands(n, rows, cols, n + rows + cols)
    space = abi.workspace(abi.ds_gemm_fp8_workspace_bytes(n, rows, cols))
    want = product(w, ws, x, xs)
    for _ in range(2):  # the second finds what the first left in the workspace
        y = torch.full((n, rows), math.nan, dtype=torch.float32, device="cuda")
        abi.ds_gemm_fp8(w, ws, x, xs, y, space)
        assert abi.ds_workspace_error(space) == 0
        close(y, *want, cols)
