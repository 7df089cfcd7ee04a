"""ctypes binding of ``libdecodestep.so`` (declared in ``include/decode_step.h``).

Argument marshalling only: every function here passes pointers and sizes to
the C ABI and raises :class:`DecodeStepError` on a non-OK status.  Importing
this module fails loudly when the library has not been built — there is no
fallback path.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdecodestep.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libdecodestep.so is not built (run `python -c 'import __graft_entry__ as g; g.build()'` "
                      "or `python -m autoregressive_decode_step_gb300.build`)")

lib = ctypes.CDLL(LIB_PATH)

# ------------------------------------------------------------------ constants
DS_OK = 560
DS_EMPTY_DIMENSION = 561
DS_A_LENGTH_MISMATCH = 562
DS_B_LENGTH_MISMATCH = 563
DS_DIMENSION_TOO_LARGE = 564
DS_CODE_OUT_OF_RANGE = 565
DS_CACHE_LENGTH_MISMATCH = 566
DS_NEW_LENGTH_MISMATCH = 567
DS_LOGITS_LENGTH_MISMATCH = 568
DS_GEMV_A_LENGTH_MISMATCH = 569
DS_GEMV_X_LENGTH_MISMATCH = 570
DS_CACHE_CAPACITY_EXCEEDED = 571
DS_BAD_DTYPE = 572
DS_CUDA_ERROR = 573
DS_WORKSPACE_TOO_SMALL = 574
DS_BAD_SAMPLING_PARAM = 575
DS_TOKEN_OUT_OF_RANGE = 576
DS_BAD_ARGUMENT = 577
DS_MAX_DIM = 1 << 24
DS_F32, DS_BF16, DS_E4M3 = 0, 1, 2
DS_ROPE_HALF_SPLIT, DS_ROPE_INTERLEAVED = 0, 1
DS_ERR_TOKEN_RANGE, DS_ERR_POSITION, DS_ERR_WAIT_TIMEOUT, DS_ERR_SAMPLING = 1, 2, 4, 8
DS_ERR_NO_BLOCKS = 16
DS_STEP_ADVANCE = 1
DS_STEP_PHASE_TIMES = 2
DS_STEP_TRACE = 4
KIND_NAMES = ["embed", "qkv", "attention", "o_proj", "gate_up", "down", "head", "sample"]

P = ctypes.c_void_p
I32 = ctypes.c_int32
I64 = ctypes.c_int64
SZ = ctypes.c_size_t
F32 = ctypes.c_float
F64 = ctypes.c_double


class ModelConfig(ctypes.Structure):
    _fields_ = [("vocab", I32), ("d", I32), ("n_layer", I32), ("n_qh", I32), ("n_kvh", I32),
                ("head_dim", I32), ("ff", I32), ("rope_layout", I32), ("rope_base", F64), ("eps", F32),
                ("tied", I32), ("w_dtype", I32), ("kv_dtype", I32), ("max_seqs", I32), ("max_ctx", I32),
                ("rope_factor", F64), ("rope_low_freq_factor", F64), ("rope_high_freq_factor", F64),
                ("rope_orig_max_pos", F64)]


class ModelWeights(ctypes.Structure):
    _fields_ = [("emb", P), ("out", P), ("final_norm", P), ("n1", P), ("wqkv", P), ("wo", P), ("n2", P),
                ("wgu", P), ("wd", P), ("q_norm", P), ("k_norm", P)]


class KVCache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("rows", I64), ("block_tokens", I32), ("max_blocks", I32),
                ("block_table", P)]


class Sampling(ctypes.Structure):
    _fields_ = [("temperature", F32), ("top_k", I32), ("top_p", F32)]


class SchedConfig(ctypes.Structure):
    _fields_ = [("n_blocks", I32), ("block_tokens", I32), ("max_blocks", I32), ("max_running", I32),
                ("chunk", I32), ("headroom_blocks", I32)]


class SchedRow(ctypes.Structure):
    _fields_ = [("request", I64), ("slot", I32), ("offset", I32), ("count", I32), ("decode", I32),
                ("yields", I32)]


def _sig(name, res, *args):
    f = getattr(lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("ds_status_name", ctypes.c_char_p, ctypes.c_int)
_sig("ds_residual_dims_check", ctypes.c_int, I64, I64, I64)
_sig("ds_workspace_error", ctypes.c_int, P, P, P)
_sig("ds_device_sm_count", ctypes.c_int)
_sig("ds_gemv_workspace_bytes", SZ, I64, I64, ctypes.c_int)
_sig("ds_gemv_transposed", ctypes.c_int, P, I64, ctypes.c_int, P, I64, I64, I64, P, I64, P, SZ, P)
_sig("ds_gemv", ctypes.c_int, P, I64, ctypes.c_int, P, I64, I64, I64, P, I64, P)
_sig("ds_gemm_workspace_bytes", SZ, I64, I64, I64)
_sig("ds_decode_steps", ctypes.c_int, P, P, P, P, ctypes.c_int, P, P, ctypes.c_uint, P)
_sig("ds_step_seq", ctypes.c_int, P, P, P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P, P)
_sig("ds_sched_create", ctypes.c_int, ctypes.POINTER(SchedConfig), P)
_sig("ds_sched_destroy", None, P)
_sig("ds_sched_submit", ctypes.c_int, P, I64, I32, I32)
_sig("ds_sched_plan", ctypes.c_int, P, P, I32, P, P, P, P)
_sig("ds_sched_commit", ctypes.c_int, P, P, I32)
_sig("ds_sched_stats", ctypes.c_int, P, P)
_sig("ds_sched_generated", I64, P, I64)
_sig("ds_gemm_transposed", ctypes.c_int, P, I64, P, I64, I64, I64, I64, P, I64, P, SZ, P)
_sig("ds_gemm", ctypes.c_int, P, I64, P, I64, I64, I64, I64, P, I64, P, SZ, P)
_sig("ds_fp8_quantize", ctypes.c_int, P, I64, ctypes.c_int, I64, I64, I64, ctypes.c_int, P, I64, I64, P, I64, P)
_sig("ds_gemm_fp8_workspace_bytes", SZ, I64, I64, I64)
_sig("ds_gemm_fp8", ctypes.c_int, P, I64, I64, P, I64, P, I64, I64, P, I64, I64, I64, I64, P, I64, ctypes.c_int, I64, P,
     SZ, P)
_sig("ds_moe_layer_workspace_bytes", SZ, I64, I64, I64, ctypes.c_int, ctypes.c_int)
_sig("ds_moe_layer", ctypes.c_int, P, I64, ctypes.c_int, I64, I64, P, I64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
     ctypes.c_int, P, I64, P, I64, P, I64, P, I64, ctypes.c_int, I64, P, P, I64, P, P, P, SZ, P)
_sig("ds_gemv_transposed_noalloc", ctypes.c_int, P, I64, ctypes.c_int, P, I64, I64, I64, P, I64, P)
_sig("ds_gemv_transposed_noalloc_max_bytes", SZ)
_sig("ds_gemv_transposed_noalloc_error", ctypes.c_int, P, P)
_sig("ds_residual_add", ctypes.c_int, P, I64, P, I64, P, I64, P)
_sig("ds_add_rmsnorm", ctypes.c_int, P, I64, P, I64, P, I64, ctypes.c_int, F32, P, I64, I64, P)
_sig("ds_rope", ctypes.c_int, P, I64, P, I64, I64, ctypes.c_int, ctypes.c_int, ctypes.c_int, F64, ctypes.c_int, P)
_sig("ds_kv_cache_append", ctypes.c_int, P, ctypes.c_int, I64, I64, P, I64, I64, P)
_sig("ds_silu_mul", ctypes.c_int, P, I64, P, I64, P, I64, P)
_sig("ds_attention_workspace_bytes", SZ, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, I64)
_sig("ds_gqa_decode_attn", ctypes.c_int, P, P, P, ctypes.c_int, I64, P, ctypes.c_int, ctypes.c_int, P,
     ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, F32, P, P, SZ, P)
_sig("ds_paged_plan_workspace_bytes", SZ)
_sig("ds_paged_plan", ctypes.c_int, P, P, ctypes.c_int, P, I64, ctypes.c_int, I64, P, ctypes.c_int, P, P, P, P, P,
     I64, P, P, SZ, P)
_sig("ds_rope_append_workspace_bytes", SZ)
_sig("ds_rope_append", ctypes.c_int, P, I64, ctypes.c_int, I64, I64, P, ctypes.c_int, P, ctypes.c_int, ctypes.c_int,
     ctypes.c_int, ctypes.c_int, F64, ctypes.c_int, P, I64, ctypes.c_int, P, P, ctypes.c_int, I64, P, P, SZ, P)
_sig("ds_chunk_attention_workspace_bytes", SZ, ctypes.c_int, I64, ctypes.c_int, ctypes.c_int, ctypes.c_int)
_sig("ds_gqa_chunk_attn", ctypes.c_int, P, I64, ctypes.c_int, I64, P, P, ctypes.c_int, P, P, ctypes.c_int, I64, P,
     ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, F32, P, I64, P, SZ, P)
_sig("ds_argmax_workspace_bytes", SZ, ctypes.c_int, I64)
_sig("ds_greedy_argmax", ctypes.c_int, P, I64, ctypes.c_int, I64, P, P, P, SZ, P)
_sig("ds_sample_workspace_bytes", SZ, ctypes.c_int, I64)
_sig("ds_sample", ctypes.c_int, P, I64, ctypes.c_int, I64, F32, ctypes.c_int, F32, P, P, P, SZ, P)
_sig("ds_model_workspace_bytes", SZ, ctypes.POINTER(ModelConfig))
_sig("ds_model_create", ctypes.c_int, ctypes.POINTER(ModelConfig), ctypes.POINTER(ModelWeights), P, SZ,
     ctypes.POINTER(P))
_sig("ds_model_destroy", None, P)
_sig("ds_model_workspace", P, P)
_sig("ds_decode_step", ctypes.c_int, P, ctypes.POINTER(KVCache), P, P, ctypes.c_int, ctypes.POINTER(Sampling),
     P, P, P, ctypes.c_uint, P)
_sig("ds_step_graph_create", ctypes.c_int, P, ctypes.POINTER(KVCache), P, P, ctypes.c_int,
     ctypes.POINTER(Sampling), P, P, P, ctypes.c_uint, P, ctypes.POINTER(P))
_sig("ds_step_graph_launch", ctypes.c_int, P, P)
_sig("ds_step_graph_destroy", None, P)
_sig("ds_model_phase_times", ctypes.c_int, P, P, ctypes.c_int, ctypes.POINTER(ctypes.c_int), P)
_sig("ds_model_trace", ctypes.c_int, P, P, SZ, ctypes.POINTER(SZ), ctypes.POINTER(ctypes.c_int), P)
_sig("ds_decode_kernel_time", ctypes.c_int, P, ctypes.POINTER(KVCache), P, P, ctypes.c_int, ctypes.c_int,
     ctypes.POINTER(ctypes.c_float), P)
_sig("ds_decode_step_profile", ctypes.c_int, P, ctypes.POINTER(KVCache), P, P, ctypes.c_int,
     ctypes.POINTER(Sampling), P, P, P, ctypes.c_uint, ctypes.c_int, P, P, ctypes.c_int,
     ctypes.POINTER(ctypes.c_int), P)


class DecodeStepError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__("%s: %s (%d)" % (where, status_name(code), code))


def status_name(code):
    return lib.ds_status_name(int(code)).decode()


def check(code, where="decode_step"):
    if code != DS_OK:
        raise DecodeStepError(code, where)
    return code


# ------------------------------------------------------------------ marshalling
def ptr(t):
    """Device (or host) address of a tensor, or NULL for None."""
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


_DTYPE_CODES = {torch.float32: DS_F32, torch.bfloat16: DS_BF16}


def dtype_code(t):
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError("unsupported dtype %s" % t.dtype)
    return code


def stream_handle(stream=None):
    if stream is None:  # the raw handle: building a Stream object takes 3 us
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return ctypes.c_void_p(stream.cuda_stream)


def nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def workspace(nbytes_, device="cuda"):
    """A zero-filled, 256-byte-aligned workspace tensor."""
    return torch.zeros(max(int(nbytes_), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ ops
def ds_gemv_workspace_bytes(rows, cols, dtype=DS_F32):
    return lib.ds_gemv_workspace_bytes(rows, cols, dtype)


def ds_gemv_transposed(A, x, rows, cols, y, ws, stream=None):
    check(lib.ds_gemv_transposed(ptr(A), A.numel(), dtype_code(A), ptr(x), x.numel(), rows, cols, ptr(y),
                                 y.numel(), ptr(ws), nbytes(ws), stream_handle(stream)), "ds_gemv_transposed")


def ds_gemv_transposed_noalloc(A, x, rows, cols, y, stream=None):
    check(lib.ds_gemv_transposed_noalloc(ptr(A), A.numel(), dtype_code(A), ptr(x), x.numel(), rows, cols, ptr(y),
                                         y.numel(), stream_handle(stream)), "ds_gemv_transposed_noalloc")


def ds_gemv_transposed_noalloc_error(stream=None):
    """Read and clear the no-allocation area's error word (current device)."""
    word = ctypes.c_int32(0)
    check(lib.ds_gemv_transposed_noalloc_error(ctypes.byref(word), stream_handle(stream)),
          "ds_gemv_transposed_noalloc_error")
    return word.value


def ds_gemv(W, x, rows, cols, y, stream=None):
    check(lib.ds_gemv(ptr(W), W.numel(), dtype_code(W), ptr(x), x.numel(), rows, cols, ptr(y), y.numel(),
                      stream_handle(stream)), "ds_gemv")


def ds_gemm_transposed(A, X, n, rows, cols, Y, ws, stream=None):
    check(lib.ds_gemm_transposed(ptr(A), A.numel(), ptr(X), X.numel(), n, rows, cols, ptr(Y), Y.numel(), ptr(ws),
                                 nbytes(ws), stream_handle(stream)), "ds_gemm_transposed")


def ds_gemm(W, X, n, rows, cols, Y, ws, stream=None):
    check(lib.ds_gemm(ptr(W), W.numel(), ptr(X), X.numel(), n, rows, cols, ptr(Y), Y.numel(), ptr(ws), nbytes(ws),
                      stream_handle(stream)), "ds_gemm")


def ds_residual_add(a, b, out, n, stream=None):
    check(lib.ds_residual_add(ptr(a), a.numel(), ptr(b), b.numel(), ptr(out), n, stream_handle(stream)),
          "ds_residual_add")


def ds_add_rmsnorm(residual, x, w, eps, h, n, stream=None):
    check(lib.ds_add_rmsnorm(ptr(residual), residual.numel(), ptr(x), 0 if x is None else x.numel(), ptr(w),
                             w.numel(), dtype_code(w), eps, ptr(h), h.numel(), n, stream_handle(stream)),
          "ds_add_rmsnorm")


def ds_rope(q, k, pos, n_qh, n_kh, head_dim, base, layout, stream=None):
    check(lib.ds_rope(ptr(q), q.numel(), ptr(k), 0 if k is None else k.numel(), pos, n_qh, n_kh, head_dim,
                      base, layout, stream_handle(stream)), "ds_rope")


def ds_kv_cache_append(cache, capacity, cache_len, new_vals, n_new, stream=None):
    check(lib.ds_kv_cache_append(ptr(cache), dtype_code(cache), capacity, cache_len, ptr(new_vals),
                                 new_vals.numel(), n_new, stream_handle(stream)), "ds_kv_cache_append")


def ds_silu_mul(gate, up, out, n, stream=None):
    check(lib.ds_silu_mul(ptr(gate), gate.numel(), ptr(up), up.numel(), ptr(out), n, stream_handle(stream)),
          "ds_silu_mul")


def ds_attention_workspace_bytes(n_seqs, n_qh, n_kvh, head_dim, max_ctx):
    return lib.ds_attention_workspace_bytes(n_seqs, n_qh, n_kvh, head_dim, max_ctx)


def ds_gqa_decode_attn(q, k_cache, v_cache, cache_rows, block_table, max_blocks_per_seq, block_tokens, seq_lens,
                       n_seqs, n_qh, n_kvh, head_dim, scale, out, ws, stream=None):
    check(lib.ds_gqa_decode_attn(ptr(q), ptr(k_cache), ptr(v_cache), dtype_code(k_cache), cache_rows,
                                 ptr(block_table), max_blocks_per_seq, block_tokens, ptr(seq_lens), n_seqs, n_qh,
                                 n_kvh, head_dim, scale, ptr(out), ptr(ws), nbytes(ws), stream_handle(stream)),
          "ds_gqa_decode_attn")


def _elsewhere(name):
    return ValueError("%s: has to be on the workspace's device" % name)


def _i32(t, n, name, dev):
    """Address of a contiguous int32 tensor of at least n elements on device dev."""
    if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() < n:
        raise ValueError("%s: a contiguous int32 tensor of %d elements is needed" % (name, n))
    if t.get_device() != dev:  # (-1 on the host)
        raise _elsewhere(name)
    return t.data_ptr()


def _here(ws):
    """Address of a workspace, which has to be on the current device: the launch goes there."""
    if not ws.is_cuda or ws.get_device() != torch._C._cuda_getDevice():
        raise ValueError("the buffers have to be on the current CUDA device")
    return ws.data_ptr()


def _dense(t, n, name, dev):
    """Address of a contiguous tensor of at least n elements on device dev."""
    if not t.is_contiguous() or t.numel() < n:
        raise ValueError("%s: a contiguous tensor of %d elements is needed" % (name, n))
    if t.get_device() != dev:
        raise _elsewhere(name)
    return t.data_ptr()


def ds_paged_plan_workspace_bytes():
    return lib.ds_paged_plan_workspace_bytes()


def ds_paged_plan(cached_lens, new_lens, n_seqs, free_blocks, block_tokens, cache_rows, block_table,
                  max_blocks_per_seq, row_starts, seq_lens, row_seq, positions, slots, max_rows, n_taken, ws,
                  stream=None):
    """Block table entries, row starts, positions and cache slots of a ragged
    step from its lengths; free_blocks may be None (no block left)."""
    dev = ws.get_device()
    n_free = 0 if free_blocks is None else free_blocks.numel()
    check(lib.ds_paged_plan(_i32(cached_lens, n_seqs, "cached_lens", dev), _i32(new_lens, n_seqs, "new_lens", dev),
                            n_seqs, _i32(free_blocks, n_free, "free_blocks", dev) if n_free else None, n_free,
                            block_tokens, cache_rows,
                            _i32(block_table, n_seqs * max_blocks_per_seq, "block_table", dev), max_blocks_per_seq,
                            _i32(row_starts, n_seqs + 1, "row_starts", dev),
                            _i32(seq_lens, n_seqs, "seq_lens", dev), _i32(row_seq, max_rows, "row_seq", dev),
                            _i32(positions, max_rows, "positions", dev), _i32(slots, max_rows, "slots", dev), max_rows,
                            _i32(n_taken, 1, "n_taken", dev), _here(ws), nbytes(ws), stream_handle(stream)),
          "ds_paged_plan")


def ds_rope_append_workspace_bytes():
    return lib.ds_rope_append_workspace_bytes()


def ds_rope_append(qkv, row_stride, n_rows, positions, n_axes, pair_axis, n_qh, n_kvh, head_dim, rot_dim, base, layout,
                   q_out, k_cache, v_cache, cache_rows, slots, ws, stream=None):
    """Rotate a ragged step's q|k|v rows and write k and v to their slots.
    pair_axis: host uint8 numpy array of rot_dim / 2 axes, or None (one axis)."""
    if pair_axis is not None:
        if pair_axis.dtype.char != "B" or pair_axis.size < rot_dim // 2:
            raise ValueError("pair_axis: a uint8 array of rot_dim / 2 axes is needed")
        pair_axis = pair_axis.tobytes()  # (the array's .ctypes takes 2 us to build)
    if v_cache.dtype != k_cache.dtype or qkv.stride(-1) != 1:
        raise ValueError("k_cache and v_cache need one dtype, qkv's rows no gaps between elements")
    n_kv, dev = cache_rows * n_kvh * head_dim, ws.get_device()
    if qkv.get_device() != dev:
        raise _elsewhere("qkv")
    # qkv may be a view of wider rows: its reach is what the storage holds from its start on
    reach = qkv.untyped_storage().nbytes() // qkv.element_size() - qkv.storage_offset()
    check(lib.ds_rope_append(qkv.data_ptr(), reach, dtype_code(qkv), row_stride, n_rows,
                             _i32(positions, n_axes * n_rows, "positions", dev), n_axes,
                             pair_axis, n_qh, n_kvh, head_dim, rot_dim, base, layout,
                             _dense(q_out, 0, "q_out", dev), q_out.numel(), dtype_code(q_out),
                             _dense(k_cache, n_kv, "k_cache", dev), _dense(v_cache, n_kv, "v_cache", dev),
                             dtype_code(k_cache),
                             cache_rows, _i32(slots, n_rows, "slots", dev), _here(ws), nbytes(ws),
                             stream_handle(stream)), "ds_rope_append")


def ds_chunk_attention_workspace_bytes(n_seqs, n_rows, n_qh, n_kvh, head_dim):
    return lib.ds_chunk_attention_workspace_bytes(n_seqs, n_rows, n_qh, n_kvh, head_dim)


def ds_gqa_chunk_attn(q, n_rows, row_starts, seq_lens, n_seqs, k_cache, v_cache, cache_rows, block_table,
                      max_blocks_per_seq, block_tokens, n_qh, n_kvh, head_dim, scale, out, ws, stream=None):
    """Causal attention of a ragged step's rows over each sequence's blocks;
    block_table None: contiguous slots."""
    if out.dtype != q.dtype or v_cache.dtype != k_cache.dtype:
        raise ValueError("q and out, and k_cache and v_cache, need one dtype each")
    n_kv, dev = cache_rows * n_kvh * head_dim, ws.get_device()
    check(lib.ds_gqa_chunk_attn(_dense(q, 0, "q", dev), q.numel(), dtype_code(q), n_rows,
                                _i32(row_starts, n_seqs + 1, "row_starts", dev),
                                _i32(seq_lens, n_seqs, "seq_lens", dev), n_seqs,
                                _dense(k_cache, n_kv, "k_cache", dev), _dense(v_cache, n_kv, "v_cache", dev),
                                dtype_code(k_cache), cache_rows,
                                None if block_table is None else _i32(block_table, n_seqs * max_blocks_per_seq,
                                                                      "block_table", dev), max_blocks_per_seq,
                                block_tokens, n_qh, n_kvh, head_dim, scale, _dense(out, 0, "out", dev), out.numel(),
                                _here(ws), nbytes(ws), stream_handle(stream)), "ds_gqa_chunk_attn")


def _rows(t, rows, cols, dtypes, name, dev, unit=1):
    """(address, elements, row stride) of a 2-D tensor of this shape and one of
    these types whose rows have no gaps; a lone row's stride is its width in
    whole units."""
    if t.dtype not in dtypes or t.shape != (rows, cols):
        raise ValueError("%s: a tensor of shape %s of %s is needed"
                         % (name, (rows, cols), " or ".join(str(d) for d in dtypes)))
    stride, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError("%s: rows without gaps between elements are needed" % name)
    if t.get_device() != dev:
        raise _elsewhere(name)
    if rows == 1:
        stride = -(-cols // unit) * unit
    return t.data_ptr(), (rows - 1) * stride + cols, stride


_E4M3, _FLOATS = (torch.float8_e4m3fn,), (torch.float32, torch.bfloat16)


def _scales(t, shape, name, dev):
    """Address of a contiguous fp32 tensor of block scales."""
    if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: a contiguous fp32 tensor of shape %s is needed" % (name, shape))
    if t.get_device() != dev:
        raise _elsewhere(name)
    return t.data_ptr()


def ds_fp8_quantize(x, block_rows, q, scales, stream=None):
    """x [rows][cols] as e4m3 codes in q with a scale for each block_rows x 128
    (1: activations, 128: weights); the rows of x and q may be views of wider ones."""
    dev = torch._C._cuda_getDevice()
    rows, cols = x.shape
    if block_rows != 1 and block_rows != 128:
        raise DecodeStepError(DS_BAD_ARGUMENT, "ds_fp8_quantize")
    rb, kb = -(-rows // block_rows), -(-cols // 128)
    xp, xn, xs = _rows(x, rows, cols, _FLOATS, "x", dev)
    qp, qn, qs = _rows(q, rows, cols, _E4M3, "q", dev)
    sp = _scales(scales, (rb, kb), "scales", dev)
    check(lib.ds_fp8_quantize(xp, xn, dtype_code(x), xs, rows, cols, block_rows, qp, qn, qs, sp, rb * kb,
                              stream_handle(stream)), "ds_fp8_quantize")


def ds_gemm_fp8_workspace_bytes(n, rows, cols):
    return lib.ds_gemm_fp8_workspace_bytes(n, rows, cols)


def ds_gemm_fp8(W, w_scales, X, x_scales, Y, ws, stream=None):
    """Y [n][rows] = X [n][cols] W [rows][cols]^T of e4m3 codes and their block scales."""
    dev = ws.get_device()
    (rows, cols), n = W.shape, X.shape[0]
    rb, kb = -(-rows // 128), -(-cols // 128)
    wp, wn, wst = _rows(W, rows, cols, _E4M3, "W", dev, 16)
    xp, xn, xst = _rows(X, n, cols, _E4M3, "X", dev, 16)
    yp, yn, yst = _rows(Y, n, rows, _FLOATS, "Y", dev)
    check(lib.ds_gemm_fp8(wp, wn, wst, _scales(w_scales, (rb, kb), "w_scales", dev), rb * kb, xp, xn, xst,
                          _scales(x_scales, (n, kb), "x_scales", dev), n * kb, n, rows, cols, yp, yn, dtype_code(Y), yst,
                          _here(ws), nbytes(ws), stream_handle(stream)), "ds_gemm_fp8")


def ds_moe_layer_workspace_bytes(n, d, ff, n_experts, top_k):
    return lib.ds_moe_layer_workspace_bytes(n, d, ff, n_experts, top_k)


def ds_moe_layer(x, w_router, top_k, renormalize, w_gate_up, gate_up_scales, w_down, down_scales, residual, y,
                 expert_ids, expert_weights, ws, stream=None):
    """y [n][d] = (residual +) the weighted sum of top_k experts' feed-forward of x [n][d].
    w_router [experts][d], w_gate_up [experts][2][ff][d], w_down [experts][d][ff]; scales for e4m3 experts, else
    None; residual, expert_ids and expert_weights may be None."""
    dev = ws.get_device()
    n, d = x.shape
    experts, _, ff, _ = w_gate_up.shape
    if (w_router.shape != (experts, d) or w_gate_up.shape != (experts, 2, ff, d) or w_down.shape != (experts, d, ff)
            or y.shape != (n, d) or y.dtype != x.dtype or w_down.dtype != w_gate_up.dtype):
        raise ValueError("ds_moe_layer: shapes or types that do not go together")
    if residual is not None and (residual.shape != (n, d) or residual.dtype != x.dtype):
        raise ValueError("residual: x's shape and type are needed")
    e4m3 = w_gate_up.dtype == torch.float8_e4m3fn
    kb, fb = -(-d // 128), -(-ff // 128)
    for name, t in (("gate_up_scales", gate_up_scales), ("down_scales", down_scales)):
        if (t is not None) != e4m3:
            raise ValueError("%s: e4m3 experts have scales, others have none" % name)
    gs = _scales(gate_up_scales, (experts, 2, fb, kb), "gate_up_scales", dev) if e4m3 else None
    dns = _scales(down_scales, (experts, kb, fb), "down_scales", dev) if e4m3 else None
    n_scales = experts * kb * fb if e4m3 else 0
    if expert_weights is not None and expert_weights.dtype != torch.float32:
        raise ValueError("expert_weights: an fp32 tensor is needed")
    check(lib.ds_moe_layer(_dense(x, 0, "x", dev), x.numel(), dtype_code(x), n, d, _dense(w_router, 0, "w_router", dev),
                           w_router.numel(), dtype_code(w_router), experts, top_k, 1 if renormalize else 0,
                           _dense(w_gate_up, 0, "w_gate_up", dev), w_gate_up.numel(), gs, 2 * n_scales,
                           _dense(w_down, 0, "w_down", dev), w_down.numel(), dns, n_scales, DS_E4M3 if e4m3 else dtype_code(w_gate_up), ff,
                           None if residual is None else _dense(residual, 0, "residual", dev), _dense(y, 0, "y", dev),
                           y.numel(), None if expert_ids is None else _i32(expert_ids, n * top_k, "expert_ids", dev),
                           None if expert_weights is None else _dense(expert_weights, n * top_k, "expert_weights", dev),
                           _here(ws), nbytes(ws), stream_handle(stream)), "ds_moe_layer")


def ds_argmax_workspace_bytes(n_rows, n):
    return lib.ds_argmax_workspace_bytes(n_rows, n)


def ds_greedy_argmax(logits, n_rows, n, ids, max_logit, ws, stream=None):
    check(lib.ds_greedy_argmax(ptr(logits), logits.numel(), n_rows, n, ptr(ids), ptr(max_logit), ptr(ws),
                               nbytes(ws), stream_handle(stream)), "ds_greedy_argmax")


def ds_sample_workspace_bytes(n_rows, n):
    return lib.ds_sample_workspace_bytes(n_rows, n)


def ds_sample(logits, n_rows, n, temperature, top_k, top_p, u, ids, ws, stream=None):
    check(lib.ds_sample(ptr(logits), logits.numel(), n_rows, n, temperature, top_k, top_p, ptr(u), ptr(ids),
                        ptr(ws), nbytes(ws), stream_handle(stream)), "ds_sample")


def ds_workspace_error(ws, stream=None):
    word = ctypes.c_int32(0)
    check(lib.ds_workspace_error(ptr(ws), ctypes.byref(word), stream_handle(stream)), "ds_workspace_error")
    return word.value
