"""Edges of the 8-bit projections and the experts."""
import pytest
import torch

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
