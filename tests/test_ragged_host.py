"""Refusals of the ragged-step operators (ds_paged_plan, ds_rope_append,
ds_gqa_chunk_attn) on the host, without a GPU: every call below returns a
status before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def abi():
    from autoregressive_decode_step_gb300 import build
    build.build()
    from autoregressive_decode_step_gb300 import abi as A
    return A


FAKE = 0x10000      # never dereferenced
FAR = 0x40000000    # a second buffer, clear of the first
NAN, INF = float("nan"), float("inf")


def plan(abi, **kw):
    a = dict(cached=FAKE, new=FAKE, n_seqs=4, free=FAKE, n_free=8, bt=16, cache_rows=1024, table=FAKE, width=8,
             starts=FAKE, lens=FAKE, row_seq=FAKE, positions=FAKE, slots=FAKE, rows=64, taken=FAKE, ws=FAKE,
             ws_bytes=256)
    a.update(kw)
    return abi.lib.ds_paged_plan(a["cached"], a["new"], a["n_seqs"], a["free"], a["n_free"], a["bt"], a["cache_rows"],
                                 a["table"], a["width"], a["starts"], a["lens"], a["row_seq"], a["positions"],
                                 a["slots"], a["rows"], a["taken"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("change,code", [
    (dict(n_seqs=0), "DS_EMPTY_DIMENSION"), (dict(bt=0), "DS_EMPTY_DIMENSION"), (dict(rows=0), "DS_EMPTY_DIMENSION"),
    (dict(n_free=-1), "DS_EMPTY_DIMENSION"), (dict(width=0), "DS_EMPTY_DIMENSION"),
    (dict(cache_rows=0), "DS_EMPTY_DIMENSION"),
    (dict(n_seqs=4097), "DS_DIMENSION_TOO_LARGE"), (dict(rows=(1 << 24) + 1), "DS_DIMENSION_TOO_LARGE"),
    (dict(width=1 << 21), "DS_DIMENSION_TOO_LARGE"), (dict(cache_rows=(1 << 24) + 1), "DS_DIMENSION_TOO_LARGE"),
    (dict(cached=None), "DS_BAD_ARGUMENT"), (dict(free=None), "DS_BAD_ARGUMENT"), (dict(taken=None), "DS_BAD_ARGUMENT"),
    (dict(slots=None), "DS_BAD_ARGUMENT"), (dict(ws=FAKE + 8), "DS_BAD_ARGUMENT"),
    (dict(ws=None), "DS_WORKSPACE_TOO_SMALL"), (dict(ws_bytes=255), "DS_WORKSPACE_TOO_SMALL"),
])
def test_plan_refusals(abi, change, code):
    assert plan(abi, **change) == getattr(abi, code)


def rope(abi, **kw):
    a = dict(qkv=FAKE, qkv_len=10 * 6 * 64, xd=0, stride=6 * 64, rows=10, pos=FAKE, axes=1, pair=None, nq=2, nkv=2,
             hd=64, rot=64, base=1e4, layout=0, q=FAR, q_len=10 * 2 * 64, qd=0, k=FAKE, v=FAKE, kd=1, cache_rows=64,
             slots=FAKE, ws=FAKE, ws_bytes=256)
    a.update(kw)
    pair = None if a["pair"] is None else np.asarray(a["pair"], np.uint8)
    return abi.lib.ds_rope_append(a["qkv"], a["qkv_len"], a["xd"], a["stride"], a["rows"], a["pos"], a["axes"],
                                  None if pair is None else pair.ctypes.data, a["nq"], a["nkv"], a["hd"], a["rot"],
                                  a["base"], a["layout"], a["q"], a["q_len"], a["qd"], a["k"], a["v"], a["kd"],
                                  a["cache_rows"], a["slots"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=0), "DS_EMPTY_DIMENSION"), (dict(axes=0), "DS_EMPTY_DIMENSION"), (dict(nkv=0), "DS_EMPTY_DIMENSION"),
    (dict(rot=0), "DS_EMPTY_DIMENSION"), (dict(rows=(1 << 24) + 1), "DS_DIMENSION_TOO_LARGE"),
    (dict(stride=6 * 64 - 1), "DS_A_LENGTH_MISMATCH"), (dict(qkv_len=10 * 6 * 64 - 1), "DS_A_LENGTH_MISMATCH"),
    (dict(q_len=10 * 2 * 64 + 1), "DS_B_LENGTH_MISMATCH"),
    (dict(xd=2), "DS_BAD_DTYPE"), (dict(qd=7), "DS_BAD_DTYPE"), (dict(kd=-1), "DS_BAD_DTYPE"),
    (dict(layout=2), "DS_BAD_DTYPE"),
    (dict(rot=63), "DS_BAD_ARGUMENT"), (dict(rot=66), "DS_BAD_ARGUMENT"), (dict(axes=9), "DS_BAD_ARGUMENT"),
    (dict(base=0.0), "DS_BAD_ARGUMENT"), (dict(base=NAN), "DS_BAD_ARGUMENT"), (dict(base=INF), "DS_BAD_ARGUMENT"),
    (dict(axes=3), "DS_BAD_ARGUMENT"), (dict(axes=3, pair=[0] * 31 + [3]), "DS_BAD_ARGUMENT"),
    (dict(q=FAKE + 4 * 10 * 6 * 64 - 4), "DS_BAD_ARGUMENT"), (dict(k=None), "DS_BAD_ARGUMENT"),
    (dict(slots=None), "DS_BAD_ARGUMENT"), (dict(pos=None), "DS_BAD_ARGUMENT"),
    (dict(ws=None), "DS_WORKSPACE_TOO_SMALL"), (dict(ws_bytes=8), "DS_WORKSPACE_TOO_SMALL"),
    (dict(ws=FAKE + 16), "DS_BAD_ARGUMENT"),
])
def test_rope_append_refusals(abi, change, code):
    assert rope(abi, **change) == getattr(abi, code)


def test_rope_append_refuses_heads_wider_than_256(abi):
    assert rope(abi, hd=260, rot=260, stride=6 * 260, qkv_len=10 * 6 * 260, q_len=10 * 2 * 260) == abi.DS_BAD_ARGUMENT


def attn(abi, **kw):
    a = dict(q=FAKE, q_len=10 * 8 * 64, qd=1, rows=10, starts=FAKE, lens=FAKE, n_seqs=2, k=FAKE, v=FAKE, kd=1,
             cache_rows=1024, table=FAKE, width=8, bt=16, nq=8, nkv=2, hd=64, scale=0.125, out=FAR, out_len=10 * 8 * 64,
             ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return abi.lib.ds_gqa_chunk_attn(a["q"], a["q_len"], a["qd"], a["rows"], a["starts"], a["lens"], a["n_seqs"],
                                     a["k"], a["v"], a["kd"], a["cache_rows"], a["table"], a["width"], a["bt"],
                                     a["nq"], a["nkv"], a["hd"], a["scale"], a["out"], a["out_len"], a["ws"],
                                     a["ws_bytes"], None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=0), "DS_EMPTY_DIMENSION"), (dict(n_seqs=0), "DS_EMPTY_DIMENSION"), (dict(bt=0), "DS_EMPTY_DIMENSION"),
    (dict(width=0), "DS_EMPTY_DIMENSION"), (dict(cache_rows=0), "DS_EMPTY_DIMENSION"),
    (dict(rows=(1 << 24) + 1), "DS_DIMENSION_TOO_LARGE"), (dict(width=1 << 21), "DS_DIMENSION_TOO_LARGE"),
    (dict(qd=2), "DS_BAD_DTYPE"), (dict(kd=3), "DS_BAD_DTYPE"),
    (dict(nq=7), "DS_BAD_ARGUMENT"), (dict(hd=66), "DS_BAD_ARGUMENT"), (dict(hd=260), "DS_BAD_ARGUMENT"),
    (dict(scale=0.0), "DS_BAD_ARGUMENT"), (dict(scale=-1.0), "DS_BAD_ARGUMENT"), (dict(scale=NAN), "DS_BAD_ARGUMENT"),
    (dict(scale=INF), "DS_BAD_ARGUMENT"),
    (dict(q_len=10 * 8 * 64 - 1), "DS_A_LENGTH_MISMATCH"), (dict(out_len=10 * 8 * 64 + 1), "DS_B_LENGTH_MISMATCH"),
    (dict(q=None), "DS_BAD_ARGUMENT"), (dict(starts=None), "DS_BAD_ARGUMENT"), (dict(k=FAKE + 8), "DS_BAD_ARGUMENT"),
    (dict(out=FAR + 2), "DS_BAD_ARGUMENT"), (dict(out=FAKE + 16), "DS_BAD_ARGUMENT"),
    (dict(table=None, cache_rows=255), "DS_CACHE_CAPACITY_EXCEEDED"),
    (dict(cache_rows=15), "DS_CACHE_CAPACITY_EXCEEDED"),
    (dict(ws=None), "DS_WORKSPACE_TOO_SMALL"), (dict(ws_bytes=256), "DS_WORKSPACE_TOO_SMALL"),
    (dict(ws=FAKE + 64), "DS_BAD_ARGUMENT"),
])
def test_chunk_attention_refusals(abi, change, code):
    assert attn(abi, **change) == getattr(abi, code)


def test_chunk_attention_workspace_bytes(abi):
    f = abi.lib.ds_chunk_attention_workspace_bytes
    assert f(1, 1, 32, 8, 128) > 256
    assert f(1, 256, 32, 8, 128) >= f(1, 8, 32, 8, 128)
    for bad in [(0, 1, 32, 8, 128), (1, 0, 32, 8, 128), (1, 1, 30, 8, 128), (1, 1, 4, 8, 128), (1, 1, 32, 8, 0),
                (1, 1, 32, 8, 257)]:
        assert f(*bad) == 0


def test_the_binding_refuses_other_integer_types_and_strides(abi):
    t32 = torch.zeros(8, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):  # int64 lengths
        abi.ds_paged_plan(t32.long(), t32, 1, t32, 16, 128, t32, 8, t32, t32, t32, t32, t32, 8, t32, ws, stream=0)
    with pytest.raises(ValueError):  # every second element
        abi.ds_paged_plan(t32, torch.zeros(16, dtype=torch.int32)[::2], 8, t32, 16, 128, t32, 1, t32, t32, t32, t32,
                          t32, 8, t32, ws, stream=0)
    x = torch.zeros(2, 6 * 64)
    with pytest.raises(ValueError):  # an axis map of the wrong type
        abi.ds_rope_append(x, 6 * 64, 2, t32, 1, np.zeros(32, np.int64), 2, 2, 64, 64, 1e4, 0, torch.zeros(2, 128),
                           torch.zeros(4, 128), torch.zeros(4, 128), 4, t32, ws, stream=0)
    q = torch.zeros(1, 8 * 64)
    kv = torch.zeros(16, 2 * 64)
    with pytest.raises(ValueError):  # out of another type than q
        abi.ds_gqa_chunk_attn(q, 1, t32, t32, 1, kv, kv, 16, None, 1, 16, 8, 2, 64, 0.125, q.bfloat16(), ws, stream=0)
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_the_binding_refuses_a_workspace_that_is_not_on_the_device(abi):
    t32 = torch.zeros(64, dtype=torch.int32)
    with pytest.raises(ValueError):
        abi.ds_paged_plan(t32, t32, 1, t32, 16, 128, t32, 8, t32, t32, t32, t32, t32, 8, t32,
                          torch.zeros(256, dtype=torch.uint8), stream=None)


@pytest.mark.parametrize("out,other", [
    ("lens", "cached"), ("lens", "new"), ("starts", "cached"), ("table", "free"), ("taken", "free"),
    ("positions", "slots"), ("row_seq", "positions"), ("lens", "starts"),
])
def test_plan_refuses_outputs_that_overlap(abi, out, other):
    names = ["cached", "new", "free", "table", "starts", "lens", "row_seq", "positions", "slots", "taken"]
    at = {n: FAKE + 0x1000 * i for i, n in enumerate(names)}
    at[out] = at[other] + 4  # (n_taken: the second free block; else all but the first element)
    assert plan(abi, **at) == abi.DS_BAD_ARGUMENT


@pytest.mark.parametrize("change", [
    dict(v=0x50000000 + 64 * 2 * 64 * 2 - 16),             # the caches' ends
    dict(k=FAKE + 4 * 10 * 6 * 64 - 16),                   # the last row's end
    dict(v=FAR + 4 * 10 * 2 * 64 - 16),                    # q_out's end
    dict(q=FAKE + 4 * 10 * 6 * 64 - 16, qkv_len=1 << 20),  # the rows' end, in a longer buffer
])
def test_rope_append_refuses_outputs_that_overlap(abi, change):
    assert rope(abi, **dict(dict(k=0x50000000, v=0x60000000), **change)) == abi.DS_BAD_ARGUMENT
