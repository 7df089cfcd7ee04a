"""The 8-bit projections and the experts as a decoder layer uses them: norm,
quantisation, q|k|v, rotation and cache, attention, quantisation, o, residual
and norm, experts, for a ragged step of three requests, eagerly and as a graph."""
import math

import pytest
import torch

from tests.test_gpu_fp8 import close, product, quantized, same_codes
from tests.test_gpu_moe import Layer

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
D, NQ, NKV, HD, FF, EXPERTS, K, BT = 512, 4, 2, 64, 208, 8, 2, 8
NEW, CACHED = [1, 5, 3], [11, 0, 7]
ROWS, WIDTH, BLOCKS = sum(NEW), 3, 12


@pytest.fixture(scope="module")
def abi():
    from autoregressive_decode_step_gb300 import build
    build.build()
    from autoregressive_decode_step_gb300 import abi as A
    return A


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """A layer's weights, the buffers of a step and the step itself."""

    def __init__(self, abi, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.abi = abi

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=g, device="cuda") / math.sqrt(cols)
            q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda").view(E4M3)
            s = torch.empty(-(-rows // 128), -(-cols // 128), device="cuda")
            abi.ds_fp8_quantize(w, 128, q, s)
            return q, s

        self.qkv_w, self.qkv_s = weight((NQ + 2 * NKV) * HD, D)
        self.o_w, self.o_s = weight(D, NQ * HD)
        self.moe = Layer(ROWS, D, FF, EXPERTS, K, w=E4M3, seed=seed)
        self.n1, self.n2 = torch.ones(D, device="cuda"), torch.rand(D, generator=g, device="cuda") + 0.5

        def rows(*shape, dtype=torch.float32):
            return torch.zeros(*shape, dtype=dtype, device="cuda")

        def codes(cols):
            return rows(ROWS, cols, dtype=torch.uint8).view(E4M3), rows(ROWS, -(-cols // 128))

        self.x, self.h, self.h2, self.y = (rows(ROWS, D) for _ in range(4))
        self.res, self.qkv, self.o = rows(ROWS, D), rows(ROWS, (NQ + 2 * NKV) * HD), rows(ROWS, D)
        self.q, self.att = rows(ROWS, NQ * HD), rows(ROWS, NQ * HD)
        self.hq, self.hs = codes(D)
        self.aq, self.as_ = codes(NQ * HD)
        self.k = torch.randn(BLOCKS * BT, NKV * HD, generator=g, device="cuda").bfloat16()
        self.v = torch.randn(BLOCKS * BT, NKV * HD, generator=g, device="cuda").bfloat16()
        self.table = i32(*torch.randperm(BLOCKS, generator=torch.Generator().manual_seed(seed))[:3 * WIDTH].tolist())
        pos = [c + i for n, c in zip(NEW, CACHED) for i in range(n)]
        seq = [s for s, n in enumerate(NEW) for _ in range(n)]
        self.pos, self.starts = i32(*pos), i32(0, *[sum(NEW[:i + 1]) for i in range(3)])
        self.lens = i32(*[n + c for n, c in zip(NEW, CACHED)])
        t = self.table.tolist()
        self.slots = i32(*[t[s * WIDTH + p // BT] * BT + p % BT for s, p in zip(seq, pos)])
        self.ids, self.p = rows(ROWS, K, dtype=torch.int32), rows(ROWS, K)
        self.ws = [abi.workspace(b) for b in (
            max(abi.ds_gemm_fp8_workspace_bytes(ROWS, (NQ + 2 * NKV) * HD, D), abi.ds_gemm_fp8_workspace_bytes(ROWS, D, NQ * HD)),
            256, abi.ds_chunk_attention_workspace_bytes(3, ROWS, NQ, NKV, HD),
            abi.ds_moe_layer_workspace_bytes(ROWS, D, FF, EXPERTS, K))]

    def run(self):
        abi, m = self.abi, self.moe
        self.res.copy_(self.x)
        for r in range(ROWS):
            abi.ds_add_rmsnorm(self.res[r], None, self.n1, 1e-5, self.h[r], D)
        abi.ds_fp8_quantize(self.h, 1, self.hq, self.hs)
        abi.ds_gemm_fp8(self.qkv_w, self.qkv_s, self.hq, self.hs, self.qkv, self.ws[0])
        abi.ds_rope_append(self.qkv, (NQ + 2 * NKV) * HD, ROWS, self.pos, 1, None, NQ, NKV, HD, HD, 1e4, 0, self.q, self.k,
                           self.v, BLOCKS * BT, self.slots, self.ws[1])
        abi.ds_gqa_chunk_attn(self.q, ROWS, self.starts, self.lens, 3, self.k, self.v, BLOCKS * BT, self.table, WIDTH, BT,
                              NQ, NKV, HD, HD ** -0.5, self.att, self.ws[2])
        abi.ds_fp8_quantize(self.att, 1, self.aq, self.as_)
        abi.ds_gemm_fp8(self.o_w, self.o_s, self.aq, self.as_, self.o, self.ws[0])
        for r in range(ROWS):
            abi.ds_add_rmsnorm(self.res[r], self.o[r], self.n2, 1e-5, self.h2[r], D)
        abi.ds_moe_layer(self.h2, m.router, K, True, m.gu, m.gs, m.dn, m.ds, self.res, self.y, self.ids, self.p, self.ws[3])

    def check(self):
        """Each stage against 64 bits on what the stage before it gave."""
        want, scale = quantized(self.h, 1)
        same_codes(self.hq, want)
        assert (torch.from_numpy(scale).cuda() == self.hs).all()
        close(self.qkv, *product(self.qkv_w, self.qkv_s, self.hq, self.hs), D)
        want, _ = quantized(self.att, 1)
        same_codes(self.aq, want)
        close(self.o, *product(self.o_w, self.o_s, self.aq, self.as_), NQ * HD)
        self.moe.x, self.moe.residual = self.h2, self.res
        want, far, ids, _ = self.moe.want()
        assert torch.equal(self.ids.long(), ids)
        assert ((self.y.double() - want).abs() <= far).all()
        assert [self.abi.ds_workspace_error(w) for w in self.ws] == [0] * 4


def test_a_layer_of_8_bit_projections_and_experts(abi):
    s = Step(abi, 3)
    s.x.copy_(torch.randn(ROWS, D, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda"))
    s.run()
    s.check()
    # an attended row's output is a mean of values of some size, so a stage that was left out shows
    assert s.att.abs().amax(1).min() > 0.01 and torch.isfinite(s.y).all()


def test_a_layer_as_a_graph_is_what_it_is_eagerly(abi):
    s = Step(abi, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            s.run()
    torch.cuda.synchronize()
    for seed in range(3):
        x = torch.randn(ROWS, D, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
        s.x.copy_(x)
        s.run()
        torch.cuda.synchronize()
        eager = s.y.clone()
        s.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.y, eager)
    s.check()
