"""More refusals of the 8-bit projections and the experts on the host: each call
returns or raises before anything is launched."""
import pytest
import torch

from tests.test_fp8_moe_host import SCALED, moe

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def abi():
    from autoregressive_decode_step_gb300 import build
    build.build()
    from autoregressive_decode_step_gb300 import abi as A
    return A


@pytest.mark.parametrize("change,code", [
    (dict(gs=SCALED["gs"]), "DS_BAD_ARGUMENT"), (dict(ds=SCALED["ds"]), "DS_BAD_ARGUMENT"),
    (dict(gs_len=SCALED["gs_len"]), "DS_GEMV_A_LENGTH_MISMATCH"), (dict(ds_len=SCALED["ds_len"]), "DS_GEMV_A_LENGTH_MISMATCH"),
])
def test_scales_of_experts_that_have_none_are_refused(abi, change, code):
    assert moe(abi, **change) == getattr(abi, code)


@pytest.mark.parametrize("which", ["gate_up_scales", "down_scales"])
def test_the_binding_refuses_scales_of_experts_that_have_none(abi, which):
    gu, dn = torch.zeros(3, 2, 16, 32, dtype=torch.bfloat16), torch.zeros(3, 32, 16, dtype=torch.bfloat16)
    scales = dict(gate_up_scales=torch.ones(3, 2, 1, 1), down_scales=torch.ones(3, 1, 1))
    a = dict(gate_up_scales=None, down_scales=None)
    a[which] = scales[which]
    with pytest.raises(ValueError, match=which):
        abi.ds_moe_layer(torch.zeros(2, 32), torch.zeros(3, 32), 2, True, gu, a["gate_up_scales"], dn, a["down_scales"], None,
                         torch.zeros(2, 32), None, None, torch.zeros(256, dtype=torch.uint8), stream=0)


@pytest.mark.parametrize("which", ["gate_up_scales", "down_scales"])
def test_the_binding_refuses_e4m3_experts_without_scales(abi, which):
    gu, dn = torch.zeros(3, 2, 16, 32, dtype=torch.uint8).view(E4M3), torch.zeros(3, 32, 16, dtype=torch.uint8).view(E4M3)
    a = dict(gate_up_scales=torch.ones(3, 2, 1, 1), down_scales=torch.ones(3, 1, 1))
    a[which] = None
    with pytest.raises(ValueError, match=which):
        abi.ds_moe_layer(torch.zeros(2, 32), torch.zeros(3, 32), 2, True, gu, a["gate_up_scales"], dn, a["down_scales"], None,
                         torch.zeros(2, 32), None, None, torch.zeros(256, dtype=torch.uint8), stream=0)
