"""Refusals of the 8-bit projections and the mixture-of-experts layer on the
host, without a GPU: every call below returns a status before anything is
launched, each for one reason."""
import pytest
import torch

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def abi():
    from autoregressive_decode_step_gb300 import build
    build.build()
    from autoregressive_decode_step_gb300 import abi as A
    return A


# addresses that nothing reads, far apart
A0, B0, C0, D0, E0, F0, G0, H0 = (0x100000000 * (i + 1) for i in range(8))


def quantize(abi, **kw):
    a = dict(x=A0, x_len=9 * 320 + 300, xd=0, xs=320, rows=10, cols=300, br=1, q=B0, q_len=9 * 304 + 300, qs=304, s=C0,
             s_len=10 * 3)
    a.update(kw)
    return abi.lib.ds_fp8_quantize(a["x"], a["x_len"], a["xd"], a["xs"], a["rows"], a["cols"], a["br"], a["q"],
                                   a["q_len"], a["qs"], a["s"], a["s_len"], None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=0), "DS_EMPTY_DIMENSION"), (dict(cols=0), "DS_EMPTY_DIMENSION"),
    (dict(rows=(1 << 24) + 1), "DS_DIMENSION_TOO_LARGE"), (dict(xs=(1 << 24) + 1), "DS_DIMENSION_TOO_LARGE"),
    (dict(qs=(1 << 24) + 1), "DS_DIMENSION_TOO_LARGE"),
    (dict(xd=2), "DS_BAD_DTYPE"), (dict(xd=-1), "DS_BAD_DTYPE"),
    (dict(br=64), "DS_BAD_ARGUMENT"), (dict(br=0), "DS_BAD_ARGUMENT"),
    (dict(xs=299, x_len=1 << 20), "DS_A_LENGTH_MISMATCH"), (dict(x_len=9 * 320 + 299), "DS_A_LENGTH_MISMATCH"),
    (dict(qs=299, q_len=1 << 20), "DS_B_LENGTH_MISMATCH"), (dict(q_len=9 * 304 + 299), "DS_B_LENGTH_MISMATCH"),
    (dict(s_len=29), "DS_B_LENGTH_MISMATCH"), (dict(br=128), "DS_B_LENGTH_MISMATCH"),
    (dict(x=None), "DS_BAD_ARGUMENT"), (dict(q=None), "DS_BAD_ARGUMENT"), (dict(s=None), "DS_BAD_ARGUMENT"),
    (dict(x=A0 + 2), "DS_BAD_ARGUMENT"), (dict(x=A0 + 1, xd=1), "DS_BAD_ARGUMENT"), (dict(s=C0 + 2), "DS_BAD_ARGUMENT"),
    (dict(q=A0 + 4 * (9 * 320 + 300) - 1), "DS_BAD_ARGUMENT"),   # the last value of x
    (dict(s=B0 + 9 * 304 + 296), "DS_BAD_ARGUMENT"),             # the last codes
    (dict(s=A0), "DS_BAD_ARGUMENT"),
])
def test_quantize_refusals(abi, change, code):
    assert quantize(abi, **change) == getattr(abi, code)


def gemm(abi, **kw):
    a = dict(w=A0, w_len=999 * 320 + 300, ws=320, wsc=B0, wsc_len=8 * 3, x=C0, x_len=4 * 304 + 300, xs=304, xsc=D0,
             xsc_len=5 * 3, n=5, rows=1000, cols=300, y=E0, y_len=4 * 1001 + 1000, yd=0, ys=1001, sp=F0, sp_len=1 << 30)
    a.update(kw)
    return abi.lib.ds_gemm_fp8(a["w"], a["w_len"], a["ws"], a["wsc"], a["wsc_len"], a["x"], a["x_len"], a["xs"], a["xsc"],
                               a["xsc_len"], a["n"], a["rows"], a["cols"], a["y"], a["y_len"], a["yd"], a["ys"], a["sp"],
                               a["sp_len"], None)


@pytest.mark.parametrize("change,code", [
    (dict(n=0), "DS_EMPTY_DIMENSION"), (dict(rows=0), "DS_EMPTY_DIMENSION"), (dict(cols=-1), "DS_EMPTY_DIMENSION"),
    (dict(n=(1 << 24) + 1), "DS_DIMENSION_TOO_LARGE"), (dict(ws=(1 << 24) + 16), "DS_DIMENSION_TOO_LARGE"),
    (dict(ys=(1 << 24) + 1), "DS_DIMENSION_TOO_LARGE"),
    (dict(yd=2), "DS_BAD_DTYPE"), (dict(yd=7), "DS_BAD_DTYPE"),
    (dict(w_len=999 * 320 + 299), "DS_GEMV_A_LENGTH_MISMATCH"), (dict(ws=288, w_len=1 << 30), "DS_GEMV_A_LENGTH_MISMATCH"),
    (dict(wsc_len=23), "DS_GEMV_A_LENGTH_MISMATCH"), (dict(x_len=4 * 304 + 299), "DS_GEMV_X_LENGTH_MISMATCH"),
    (dict(xs=288, x_len=1 << 30), "DS_GEMV_X_LENGTH_MISMATCH"), (dict(xsc_len=16), "DS_GEMV_X_LENGTH_MISMATCH"),
    (dict(ys=999, y_len=1 << 30), "DS_A_LENGTH_MISMATCH"), (dict(y_len=4 * 1001 + 999), "DS_A_LENGTH_MISMATCH"),
    (dict(w=None), "DS_BAD_ARGUMENT"), (dict(x=None), "DS_BAD_ARGUMENT"), (dict(y=None), "DS_BAD_ARGUMENT"),
    (dict(wsc=None), "DS_BAD_ARGUMENT"), (dict(xsc=None), "DS_BAD_ARGUMENT"),
    (dict(w=A0 + 8), "DS_BAD_ARGUMENT"), (dict(x=C0 + 4), "DS_BAD_ARGUMENT"),
    (dict(ws=321, w_len=1 << 30), "DS_BAD_ARGUMENT"), (dict(xs=312, x_len=1 << 30), "DS_BAD_ARGUMENT"),
    (dict(y=E0 + 2), "DS_BAD_ARGUMENT"), (dict(wsc=B0 + 1), "DS_BAD_ARGUMENT"), (dict(xsc=D0 + 2), "DS_BAD_ARGUMENT"),
    (dict(y=A0 + 999 * 320 + 296), "DS_BAD_ARGUMENT"), (dict(y=D0 + 56), "DS_BAD_ARGUMENT"),  # an input's end
    (dict(y=C0 - 4 * (4 * 1001 + 999)), "DS_BAD_ARGUMENT"),                                   # its own end
    (dict(sp=None), "DS_WORKSPACE_TOO_SMALL"), (dict(sp_len=256), "DS_WORKSPACE_TOO_SMALL"),
    (dict(sp=F0 + 16), "DS_BAD_ARGUMENT"),
])
def test_gemm_fp8_refusals(abi, change, code):
    assert gemm(abi, **change) == getattr(abi, code)


def test_gemm_fp8_workspace_bytes(abi):
    f = abi.ds_gemm_fp8_workspace_bytes
    for n in (1, 16, 17, 64, 128, 129, 8192, 1 << 24):
        assert f(n, 4096, 4096) >= 256
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), ((1 << 24) + 1, 1, 1)):
        assert f(*bad) == 0
    # the answer is what the call wants
    want = f(5, 1000, 300)
    assert gemm(abi, sp_len=want - 1) == abi.DS_WORKSPACE_TOO_SMALL


def moe(abi, **kw):
    n, d, ff, e = 6, 256, 192, 4
    a = dict(x=A0, x_len=n * d, xd=0, n=n, d=d, r=B0, r_len=e * d, rd=1, e=e, k=2, norm=1, gu=C0, gu_len=e * 2 * ff * d,
             gs=None, gs_len=0, dn=D0, dn_len=e * d * ff, ds=None, ds_len=0, wd=1, ff=ff, res=None, y=E0, y_len=n * d,
             ids=F0, wts=G0, sp=H0, sp_len=1 << 40)
    a.update(kw)
    return abi.lib.ds_moe_layer(a["x"], a["x_len"], a["xd"], a["n"], a["d"], a["r"], a["r_len"], a["rd"], a["e"], a["k"],
                                a["norm"], a["gu"], a["gu_len"], a["gs"], a["gs_len"], a["dn"], a["dn_len"], a["ds"],
                                a["ds_len"], a["wd"], a["ff"], a["res"], a["y"], a["y_len"], a["ids"], a["wts"], a["sp"],
                                a["sp_len"], None)


SCALED = dict(wd=2, gs=0x900000000, gs_len=4 * 2 * 2 * 2, ds=0xa00000000, ds_len=4 * 2 * 2)


@pytest.mark.parametrize("change,code", [
    (dict(n=0), "DS_EMPTY_DIMENSION"), (dict(d=0), "DS_EMPTY_DIMENSION"), (dict(ff=0), "DS_EMPTY_DIMENSION"),
    (dict(e=0), "DS_EMPTY_DIMENSION"), (dict(k=0), "DS_EMPTY_DIMENSION"),
    (dict(n=257), "DS_DIMENSION_TOO_LARGE"), (dict(e=513), "DS_DIMENSION_TOO_LARGE"), (dict(k=17), "DS_DIMENSION_TOO_LARGE"),
    (dict(d=(1 << 24) + 16), "DS_DIMENSION_TOO_LARGE"), (dict(d=1 << 23, ff=1 << 23), "DS_DIMENSION_TOO_LARGE"),
    (dict(xd=2), "DS_BAD_DTYPE"), (dict(rd=2), "DS_BAD_DTYPE"), (dict(wd=0), "DS_BAD_DTYPE"), (dict(wd=3), "DS_BAD_DTYPE"),
    (dict(x_len=6 * 256 - 1), "DS_GEMV_X_LENGTH_MISMATCH"), (dict(r_len=4 * 256 + 1), "DS_GEMV_A_LENGTH_MISMATCH"),
    (dict(gu_len=1), "DS_GEMV_A_LENGTH_MISMATCH"), (dict(dn_len=1), "DS_GEMV_A_LENGTH_MISMATCH"),
    (dict(SCALED, gs_len=15), "DS_GEMV_A_LENGTH_MISMATCH"), (dict(SCALED, ds_len=17), "DS_GEMV_A_LENGTH_MISMATCH"),
    (dict(y_len=1), "DS_A_LENGTH_MISMATCH"),
    (dict(k=5), "DS_BAD_ARGUMENT"),  # more than there are experts
    (dict(d=252, x_len=6 * 252, r_len=4 * 252, gu_len=4 * 2 * 192 * 252, dn_len=4 * 252 * 192, y_len=6 * 252),
     "DS_BAD_ARGUMENT"),
    (dict(SCALED, d=248, x_len=6 * 248, r_len=4 * 248, gu_len=4 * 2 * 192 * 248, dn_len=4 * 248 * 192, y_len=6 * 248),
     "DS_BAD_ARGUMENT"),  # a multiple of 8, not of 16
    (dict(x=None), "DS_BAD_ARGUMENT"), (dict(r=None), "DS_BAD_ARGUMENT"), (dict(gu=None), "DS_BAD_ARGUMENT"),
    (dict(dn=None), "DS_BAD_ARGUMENT"), (dict(y=None), "DS_BAD_ARGUMENT"),
    (dict(SCALED, gs=None), "DS_BAD_ARGUMENT"), (dict(SCALED, ds=None), "DS_BAD_ARGUMENT"),
    (dict(x=A0 + 4), "DS_BAD_ARGUMENT"), (dict(r=B0 + 2), "DS_BAD_ARGUMENT"), (dict(gu=C0 + 8), "DS_BAD_ARGUMENT"),
    (dict(dn=D0 + 8), "DS_BAD_ARGUMENT"), (dict(y=E0 + 2), "DS_BAD_ARGUMENT"), (dict(res=E0 + 1), "DS_BAD_ARGUMENT"),
    (dict(ids=F0 + 2), "DS_BAD_ARGUMENT"), (dict(wts=G0 + 1), "DS_BAD_ARGUMENT"),
    (dict(SCALED, gs=0x900000002), "DS_BAD_ARGUMENT"),
    (dict(y=A0 + 16), "DS_BAD_ARGUMENT"),                    # over x, not x itself
    (dict(res=E0 + 16), "DS_BAD_ARGUMENT"),                  # the residual over y
    (dict(ids=E0), "DS_BAD_ARGUMENT"), (dict(wts=F0 + 44), "DS_BAD_ARGUMENT"), (dict(y=C0 + 4), "DS_BAD_ARGUMENT"),
    (dict(wts=B0 + 4 * 256 * 2 - 4), "DS_BAD_ARGUMENT"), (dict(SCALED, ids=0xa0000003c), "DS_BAD_ARGUMENT"),
    (dict(sp=None), "DS_WORKSPACE_TOO_SMALL"), (dict(sp_len=4096), "DS_WORKSPACE_TOO_SMALL"),
    (dict(sp=H0 + 128), "DS_BAD_ARGUMENT"),
])
def test_moe_layer_refusals(abi, change, code):
    assert moe(abi, **change) == getattr(abi, code)


def test_moe_layer_workspace_bytes(abi):
    f = abi.ds_moe_layer_workspace_bytes
    assert f(1, 8, 8, 1, 1) > 256 and f(256, 4096, 14336, 512, 16) > f(64, 4096, 14336, 512, 16)
    for bad in ((0, 8, 8, 1, 1), (257, 8, 8, 1, 1), (1, 0, 8, 1, 1), (1, 8, 8, 513, 1), (1, 8, 8, 4, 17)):
        assert f(*bad) == 0
    assert moe(abi, sp_len=f(6, 256, 192, 4, 2) - 1) == abi.DS_WORKSPACE_TOO_SMALL


def test_the_binding_refuses_shapes_types_and_gaps(abi):
    codes = torch.zeros(4, 256, dtype=torch.uint8).view(E4M3)
    ws = torch.zeros(256, dtype=torch.uint8)
    x, y, one = torch.zeros(2, 256), torch.zeros(2, 4), torch.ones(1, 2)
    xs = torch.ones(2, 2)
    bad = [(codes, one, x, xs, y), (codes, one, codes[:2, ::2], torch.ones(2, 1), y), (codes, one.double(), codes[:2], xs, y),
           (codes, torch.ones(2, 2), codes[:2], xs, y), (codes, one, codes[:2], xs, torch.zeros(2, 5)),
           (codes, one, codes[:2], xs, y.half())]
    for args in bad:
        with pytest.raises(ValueError):
            abi.ds_gemm_fp8(*args, ws, stream=0)
    gu, dn = torch.zeros(3, 2, 16, 32, dtype=torch.bfloat16), torch.zeros(3, 32, 16, dtype=torch.bfloat16)
    x, r = torch.zeros(2, 32), torch.zeros(3, 32)
    for change in (dict(r=r[:2]), dict(dn=dn[:, :16]), dict(dn=dn.float()), dict(y=torch.zeros(2, 33)), dict(y=x.bfloat16()),
                   dict(res=x.bfloat16()), dict(wts=torch.zeros(2, 2, dtype=torch.float64)),
                   dict(ids=torch.zeros(2, 2, dtype=torch.int64)), dict(gu=gu.transpose(2, 3).contiguous())):
        a = dict(dict(r=r, gu=gu, dn=dn, res=None, y=torch.zeros(2, 32), ids=None, wts=None), **change)
        with pytest.raises(ValueError):
            abi.ds_moe_layer(x, a["r"], 2, True, a["gu"], None, a["dn"], None, a["res"], a["y"], a["ids"], a["wts"], ws,
                             stream=0)
