"""Host side of the ragged-step operators without a GPU: what a call would
launch, and refusals with a single reason each."""
import struct
from decimal import Decimal, getcontext

import pytest

from tests import fake_runtime

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


@pytest.mark.parametrize("base", [1e-8, 1e-3, 0.75, 1.0, 10000.0, 500000.0, 1e6, 1e30, 1.7e308])
@pytest.mark.parametrize("hd,rot", [(128, 128), (256, 256), (80, 48), (6, 2), (4, 4)])
def test_the_rotary_frequency_is_right_to_its_last_bit(tmp_path, base, hd, rot):
    """The kernel multiplies positions by base^(-2p / rot) / 2 pi as a fraction of a turn in units of 2^-64: a unit at
    most from 60 digits' answer, so a position below 2^31 leaves less than 2^-33 of a turn."""
    getcontext().prec = 80
    out = fake_runtime.run("""
        arg_bytes = %d
        assert rope(1, 1, 1, %d, %d, %r) == DS_OK
        print(launches[0][3].hex())
        """ % (4 * rot, hd, rot, base), str(tmp_path))
    turns = struct.unpack("<%dQ" % (rot // 2), bytes.fromhex(out.strip())[:4 * rot])
    for p, got in enumerate(turns):
        want = Decimal(base) ** (Decimal(-2 * p) / rot) / (2 * PI) % 1 * 2 ** 64
        off = abs(got - want)
        assert min(off, 2 ** 64 - off) <= 1, (p, got, want)


@pytest.mark.parametrize("dtype,nq,nkv", [(0, 32, 8), (1, 64, 16)])
def test_a_narrow_call_inside_a_wide_one_takes_no_shared_memory_from_it(tmp_path, dtype, nq, nkv):
    """The limit of a kernel's shared memory belongs to the kernel, not to the call: another thread's call for narrower
    rows that comes between a call's setting it and its launch must not lower it."""
    out = fake_runtime.run("""
        inner = []
        on_set_limit.append(lambda: inner.append(rope(2048, 1, 1, 128, 128, 1e4, %d)))
        shim.shim_hook(hook)
        outer = rope(2048, %d, %d, 128, 128, 1e4, %d)
        assert inner == [DS_OK] and len(launches) == 2 and launches[1][0] > 48 * 1024 > launches[0][0], launches
        print(outer == DS_OK, [l[2] for l in launches])
        """ % (dtype, nq, nkv, dtype), str(tmp_path))
    assert out.strip() == "True [0, 0]"


def test_the_chunk_attention_waits_at_no_barrier_by_what_it_read():
    """A hardware barrier has no time limit, so whether a warp goes to one must not hang on data that its neighbours may
    have read otherwise: once a bounded wait has given up, nothing orders the notes on non-finite values. Only what the
    segment says (the same words in every warp) may decide."""
    import os
    import re
    import autoregressive_decode_step_gb300 as pkg
    with open(os.path.join(os.path.dirname(pkg.__file__), "csrc", "chunk_attn_tc.cu")) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    body = src[src.index("chunk_tc_kernel(const __grid_constant__"):src.index("bool chunk_tc_supported")]
    conditions, at = [], []  # the open blocks' conditions where each barrier stands
    i = 0
    for m in re.finditer(r"[{}]|(?:named_sync|__syncthreads)\(", body):
        if m.group() == "{":
            at.append(body[i:m.start()].rsplit(";", 1)[-1])
        elif m.group() == "}":
            at.pop()
        else:
            conditions.append(" ".join(at + [body[i:m.start()].rsplit(";", 1)[-1]]))
        i = m.end()
    assert len(conditions) >= 4
    for c in conditions:
        assert not re.search(r"\b(notes|noted|bad|dead|any|busy|valid)\b", c.replace("*dead)", "")), c


class Placed:
    """What the binding looks at of a tensor, on a device of choice."""

    def __init__(self, dtype, n, device=0, width=None):
        self.dtype, self.n, self.device, self.width = dtype, n, device, width
        self.is_cuda = device >= 0

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 0x1000

    def stride(self, dim):
        return 1 if dim == -1 else self.width

    def storage_offset(self):
        return 0

    def untyped_storage(self):
        return self

    def nbytes(self):
        return self.n * self.element_size()


def _calls(abi):
    """Per operator: the tensors of a call by name, and the call."""
    import torch
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    names = "cached new free table starts lens row_seq pos slots taken"
    plan = {k: (i32, 64) for k in names.split()}
    rope = dict(qkv=(f32, 4 * 384), pos=(i32, 4), q=(f32, 4 * 128), k=(f32, 8 * 128), v=(f32, 8 * 128), slots=(i32, 4))
    attn = dict(q=(f32, 4 * 512), starts=(i32, 3), lens=(i32, 2), k=(f32, 256 * 128), v=(f32, 256 * 128),
                table=(i32, 16), out=(f32, 4 * 512))
    return {
        "ds_paged_plan": (plan, lambda t, ws: abi.ds_paged_plan(
            t["cached"], t["new"], 2, t["free"], 16, 1024, t["table"], 8, t["starts"], t["lens"], t["row_seq"],
            t["pos"], t["slots"], 16, t["taken"], ws)),
        "ds_rope_append": (rope, lambda t, ws: abi.ds_rope_append(
            t["qkv"], 384, 4, t["pos"], 1, None, 2, 2, 64, 64, 1e4, 0, t["q"], t["k"], t["v"], 8, t["slots"], ws)),
        "ds_gqa_chunk_attn": (attn, lambda t, ws: abi.ds_gqa_chunk_attn(
            t["q"], 4, t["starts"], t["lens"], 2, t["k"], t["v"], 256, t["table"], 8, 16, 8, 2, 64, 0.125, t["out"],
            ws)),
    }


@pytest.mark.parametrize("op", ["ds_paged_plan", "ds_rope_append", "ds_gqa_chunk_attn"])
def test_the_binding_refuses_tensors_that_are_not_on_the_current_device(monkeypatch, op):
    """Lengths, slots, tables or rows left on the host or on another GPU would be read by the kernel as addresses of the
    current one."""
    import torch
    from autoregressive_decode_step_gb300 import build
    build.build()
    from autoregressive_decode_step_gb300 import abi
    reached = []
    monkeypatch.setattr(abi.lib, op, lambda *a: reached.append(a) or abi.DS_OK)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    kinds, call = _calls(abi)[op]
    good = {k: Placed(*v) for k, v in kinds.items()}
    ws = Placed(torch.uint8, 1 << 20)
    call(good, ws)
    assert len(reached) == 1
    for name in list(kinds) + ["ws"]:
        for device in (-1, 1):
            moved = dict(good)
            there = Placed(torch.uint8, 1 << 20, device) if name == "ws" else Placed(*kinds[name], device)
            if name != "ws":
                moved[name] = there
            with pytest.raises(ValueError, match="device"):
                call(moved, there if name == "ws" else ws)
    everything = {k: Placed(*v, 1) for k, v in kinds.items()}  # together, but elsewhere
    with pytest.raises(ValueError, match="device"):
        call(everything, Placed(torch.uint8, 1 << 20, 1))
    assert len(reached) == 1


# Buffers of their own for every argument, so that what a case changes is its only reason; the fake runtime takes the
# place of a launch, so a check that is missing shows as a call that is accepted, with or without a GPU.
REFUSALS = """
import numpy as np
AT = {n: 0x100000000 * (i + 1) for i, n in enumerate(
    "cached new free table starts lens row_seq positions slots taken ws qkv pos q k v".split())}
NAN, INF = float("nan"), float("inf")
def plan(**kw):
    a = dict(AT, n_seqs=4, n_free=8, bt=16, cache_rows=1024, width=8, rows=64, ws_bytes=256)
    a.update(kw)
    return lib.ds_paged_plan(a["cached"], a["new"], a["n_seqs"], a["free"], a["n_free"], a["bt"], a["cache_rows"],
                             a["table"], a["width"], a["starts"], a["lens"], a["row_seq"], a["positions"], a["slots"],
                             a["rows"], a["taken"], a["ws"], a["ws_bytes"], None)
def rope(**kw):
    hd = kw.get("hd", 64)
    a = dict(AT, qkv_len=10 * 6 * hd, xd=0, stride=6 * hd, rows=10, axes=1, pair=None, nq=2, nkv=2, hd=hd,
             rot=min(hd, 256), base=1e4, layout=0, q_len=10 * 2 * hd, qd=0, kd=1, cache_rows=64, ws_bytes=256)
    a.update(kw)
    pair = None if a["pair"] is None else np.asarray(a["pair"], np.uint8)
    return lib.ds_rope_append(a["qkv"], a["qkv_len"], a["xd"], a["stride"], a["rows"], a["pos"], a["axes"],
                              None if pair is None else pair.ctypes.data, a["nq"], a["nkv"], a["hd"], a["rot"],
                              a["base"], a["layout"], a["q"], a["q_len"], a["qd"], a["k"], a["v"], a["kd"],
                              a["cache_rows"], a["slots"], a["ws"], a["ws_bytes"], None)
for op, change in CASES:
    before = len(launches)
    print(eval(op)(**eval(change)), len(launches) - before)
"""

PLAN_CASES = [
    ("dict()", 560), ("dict(n_free=0, free=None)", 560),
    ("dict(n_seqs=0)", 561), ("dict(bt=0)", 561), ("dict(rows=0)", 561), ("dict(n_free=-1)", 561),
    ("dict(width=0)", 561), ("dict(cache_rows=0)", 561), ("dict(n_seqs=4097)", 564), ("dict(rows=(1 << 24) + 1)", 564),
    ("dict(width=1 << 21)", 564), ("dict(cache_rows=(1 << 24) + 1)", 564), ("dict(n_free=(1 << 24) + 1)", 564),
    ("dict(ws=None)", "DS_WORKSPACE_TOO_SMALL"), ("dict(ws_bytes=255)", "DS_WORKSPACE_TOO_SMALL"),
    ("dict(ws=AT['ws'] + 8)", 577), ("dict(slots=AT['positions'] + 4 * 63)", 577),
    ("dict(slots=AT['positions'] + 4 * 64)", 560),  # side by side
] + [("dict(%s=None)" % n, 577) for n in
     "cached new free table starts lens row_seq positions slots taken".split()]

ROPE_CASES = [
    ("dict()", 560), ("dict(axes=3, pair=[0] * 31 + [2])", 560), ("dict(rot=62)", 560), ("dict(hd=256)", 560),
    ("dict(rows=0)", 561), ("dict(axes=0)", 561), ("dict(nkv=0)", 561), ("dict(rot=0)", 561),
    ("dict(cache_rows=0)", 561),
    ("dict(rows=(1 << 24) + 1)", 564), ("dict(cache_rows=(1 << 24) + 1)", 564),
    ("dict(stride=6 * 64 - 1)", 562), ("dict(qkv_len=10 * 6 * 64 - 1)", 562), ("dict(q_len=10 * 2 * 64 + 1)", 563),
    ("dict(xd=2)", 572), ("dict(qd=7)", 572), ("dict(kd=-1)", 572), ("dict(layout=2)", 572),
    ("dict(rot=63)", 577), ("dict(rot=66)", 577), ("dict(axes=9, pair=[0] * 32)", 577), ("dict(hd=260)", 577),
    ("dict(base=0.0)", 577), ("dict(base=-1.0)", 577), ("dict(base=NAN)", 577), ("dict(base=INF)", 577),
    ("dict(axes=3)", 577), ("dict(axes=3, pair=[0] * 31 + [3])", 577),
    ("dict(q=AT['qkv'] + 4 * 10 * 6 * 64 - 4)", 577), ("dict(q=AT['qkv'] + 4 * 10 * 6 * 64)", 560),
    ("dict(v=AT['k'] + 64 * 2 * 64 * 2 - 2)", 577), ("dict(v=AT['k'] + 64 * 2 * 64 * 2)", 560),
    ("dict(ws=None)", "DS_WORKSPACE_TOO_SMALL"), ("dict(ws_bytes=8)", "DS_WORKSPACE_TOO_SMALL"),
    ("dict(ws=AT['ws'] + 16)", 577),
] + [("dict(%s=None)" % n, 577) for n in "qkv pos q k v slots".split()]


@pytest.mark.parametrize("op,cases", [("plan", PLAN_CASES), ("rope", ROPE_CASES)])
def test_refusals_with_one_reason_each(tmp_path, op, cases):
    from autoregressive_decode_step_gb300 import build
    build.build()
    from autoregressive_decode_step_gb300 import abi
    want = [getattr(abi, c) if isinstance(c, str) else c for _, c in cases]
    out = fake_runtime.run("CASES = %r\n" % [(op, c) for c, _ in cases] + REFUSALS, str(tmp_path))
    got = [tuple(int(x) for x in line.split()) for line in out.splitlines()]
    assert len(got) == len(cases)
    for (change, _), code, (status, launched) in zip(cases, want, got):
        assert (status, launched) == (code, int(code == abi.DS_OK)), change


@pytest.mark.parametrize("hd", [64, 128])
def test_a_lost_piece_of_fp32_attention_would_show(hd):
    """The bound that the fp32 attention is held to on the GPU, on the CPU: attention with a piece of q or of the
    weights left out breaks it in one case at least, with all of them it does not."""
    from tests.test_gpu_ragged_edges import PIECE_CASES, piece_bound, piece_data, piece_reference
    worst = {}
    for smax, T in PIECE_CASES:
        q, k, v = piece_data(smax, T, 40, 8, 2, hd)
        want = piece_reference(q, k, v, T)
        for kept in ((3, 3), (2, 3), (3, 2)):
            err = (piece_reference(q, k, v, T, *kept) - want).abs().max()
            worst[kept] = max(worst.get(kept, 0), float(err) / piece_bound(smax, T))
    assert worst[3, 3] <= 0.25 and worst[2, 3] > 1.5 and worst[3, 2] > 1.5, worst
