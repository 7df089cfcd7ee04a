"""Measured calls of the 8-bit projections and of the mixture-of-experts layer.

Three operators of a decoder whose weights are e4m3 with one scale for each
block of 128 x 128, or whose feed-forward is a mixture of experts:

* ``quant``    rows (a scale per 128 values) or weights (a scale per block of
  128 x 128) in e4m3 (``ds_fp8_quantize``);
* ``product``  Y = X W^T of block-scaled e4m3 operands (``ds_gemm_fp8``);
* ``experts``  router, top-k, the chosen experts' gate, up and down products
  and their weighted sum, for few tokens (``ds_moe_layer``).

``run`` computes an operator in plain torch operations, or, with ``own`` true,
through the library.
"""
import math

import numpy as np
import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"fp32": 4, "bf16": 2, "e4m3": 1}
TINY = 2.0 ** -96  # the least maximum a block's scale is taken from


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token's activations in front of a projection (the smallest call: latency)
        dict(name="quant token 1x4096", op="quant", rows=1, cols=4096, block=1, x="fp32", pad=0),
        # a long prompt's feed-forward activations (bandwidth)
        dict(name="quant prompt 8192x14336", op="quant", rows=8192, cols=14336, block=1, x="bf16", pad=0),
        # a weight matrix laid out once at loading, odd sizes, rows apart
        dict(name="quant weights 4099x1001", op="quant", rows=4099, cols=1001, block=128, x="bf16", pad=23),
        # one user chatting: q|k|v of one token (latency, weight bytes)
        dict(name="product token 1", op="product", n=1, rows=6144, cols=4096, y="fp32"),
        # a decode batch through gate|up (weight bytes)
        dict(name="product batch 64", op="product", n=64, rows=28672, cols=4096, y="bf16"),
        # a prompt chunk through down: few tiles, a long sum
        dict(name="product chunk 256", op="product", n=256, rows=4096, cols=14336, y="fp32"),
        # a whole long prompt through gate|up (the largest call: tensor products)
        dict(name="product prompt 8192", op="product", n=8192, rows=28672, cols=4096, y="bf16"),
        # odd everything: rows, features and a last block of 8 columns, rows padded to 16 bytes
        dict(name="product ragged 333", op="product", n=333, rows=1000, cols=1416, y="fp32"),
        # one token through many small experts: 8 of 128 (latency, weight bytes)
        dict(name="experts token 1 of 128", op="experts", n=1, d=2048, ff=768, experts=128, k=8, x="fp32", w="bf16",
             norm=True, residual=True, skew=0.0),
        # a decode batch through the same experts in e4m3: all of them are read
        dict(name="experts batch 64 e4m3", op="experts", n=64, d=2048, ff=768, experts=128, k=8, x="bf16", w="e4m3",
             norm=True, residual=False, skew=0.0),
        # a decode batch through a few wide experts, fp32 activations (the largest stream of weights)
        dict(name="experts batch 64 of 8", op="experts", n=64, d=4096, ff=14336, experts=8, k=2, x="fp32", w="bf16",
             norm=True, residual=False, skew=0.0),
        # a handful of tokens that prefer the same experts, odd sizes, weights as the softmax gives them
        dict(name="experts ragged 7 of 60", op="experts", n=7, d=1000, ff=344, experts=60, k=4, x="bf16", w="bf16",
             norm=False, residual=True, skew=1.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "experts", "experts"])
    if op == "quant":
        block = rng.choice([1, 1, 128])
        return dict(op="quant", rows=_log(rng, 1, 8192), cols=_log(rng, 64, 14336), block=block,
                    x=rng.choice(["fp32", "bf16", "bf16"]) if block == 1 else "bf16", pad=rng.choice([0, 0, 8, 23]))
    if op == "product":
        return dict(op="product", n=_log(rng, 1, 8192), rows=_log(rng, 64, 28672), cols=_log(rng, 128, 4096),
                    y=rng.choice(["fp32", "bf16"]))
    experts = _log(rng, 4, 128)
    w = rng.choice(["bf16", "e4m3"])
    return dict(op="experts", n=_log(rng, 1, 64), d=16 * _log(rng, 8, 256), ff=16 * _log(rng, 8, 112), experts=experts,
                k=rng.randrange(1, min(8, experts) + 1), x=rng.choice(["fp32", "bf16"]), w=w,
                norm=rng.choice([True, False]), residual=rng.choice([True, False]), skew=rng.choice([0.0, 0.0, 1.5]))


# ----------------------------------------------------------------- prepare
def _blocks(x, br):
    """x [..., rows, cols] as [..., row blocks, br, column blocks, 128], zeros behind the ends."""
    rows, cols = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -cols % 128, 0, -rows % br))
    return x.reshape(*x.shape[:-2], x.shape[-2] // br, br, x.shape[-1] // 128, 128)


def _plain_quantize(x, br):
    """(e4m3 values, fp32 scales) of x [..., rows, cols] with a scale for each br x 128 values."""
    rows, cols = x.shape[-2:]
    b = _blocks(x.float(), br)
    top = b.abs().amax((-3, -1), keepdim=True)
    fine = top <= torch.finfo(torch.float32).max  # neither NaN nor infinite
    top = torch.where(fine, top.clamp(min=TINY), torch.full_like(top, math.nan))
    scale = top / 448
    # (448 / top) rounded, times x rounded, is at most 448 (1 + 2^-23): rounds to 448
    q = (b * (torch.full_like(top, 448) / top)).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(*x.shape[:-2], -1, b.shape[-2] * 128)[..., :rows, :cols]
    return q.contiguous().view(torch.float8_e4m3fn), scale[..., 0, :, 0].contiguous()


def _widen(q, scale, br):
    """The numbers that e4m3 values [..., rows, cols] and their scales stand for, in fp32."""
    rows, cols = q.shape[-2:]
    s = scale.repeat_interleave(br, -2)[..., :rows, :] if br > 1 else scale
    return q.float() * s.repeat_interleave(128, -1)[..., :cols]


def _rows16(q):
    """The same values in rows that are a multiple of 16 bytes apart, as the product wants them."""
    ld = -(-q.shape[1] // 16) * 16
    wide = torch.zeros(q.shape[0], ld, dtype=torch.uint8, device=q.device)
    wide[:, :q.shape[1]] = q.view(torch.uint8)
    return wide.view(torch.float8_e4m3fn)[:, :q.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    def rows_of(n, d):
        """Activations: normal values, every channel with a size of its own and a few of them large."""
        size = torch.exp(0.5 * normal(d)) * torch.where(torch.rand(d, generator=g, device="cuda") < 0.005, 8.0, 1.0)
        return normal(n, d) * size / size.square().mean().sqrt()

    if case["op"] == "quant":
        rows, cols, br = case["rows"], case["cols"], case["block"]
        if br == 1:
            x = normal(rows, cols + case["pad"], dtype=_DT[case["x"]])
            x *= torch.exp(0.5 * normal(cols + case["pad"])).to(x.dtype)
        else:
            x = normal(rows, cols + case["pad"], dtype=_DT[case["x"]]) * 0.02
        st["x"] = x[:, :cols]
        # the buffers that a serving loop keeps from step to step
        st["q"] = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        st["scales"] = torch.zeros(-(-rows // br), -(-cols // 128), device="cuda")
        nbytes = 0
    elif case["op"] == "product":
        n, rows, cols = case["n"], case["rows"], case["cols"]
        w, st["w_scales"] = _plain_quantize(normal(rows, cols) / math.sqrt(cols), 128)
        x, st["x_scales"] = _plain_quantize(rows_of(n, cols), 1)
        st["w"], st["x"] = _rows16(w), _rows16(x)
        st["y"] = torch.zeros(n, rows, dtype=_DT[case["y"]], device="cuda")
    else:
        n, d, ff, e = case["n"], case["d"], case["ff"], case["experts"]
        st["x"] = rows_of(n, d).to(_DT[case["x"]])
        router = normal(e, d) / math.sqrt(d)
        if case["skew"]:  # a direction that the tokens share makes some experts their favourites
            lean = normal(d)
            router += case["skew"] * normal(e)[:, None] * lean[None] / d
            st["x"] += lean.to(st["x"].dtype)
        st["router"] = router.to(torch.bfloat16)
        if case["w"] == "bf16":
            st["gate_up"] = normal(e, 2, ff, d, dtype=torch.bfloat16).mul_(1 / math.sqrt(d))
            st["down"] = normal(e, d, ff, dtype=torch.bfloat16).mul_(1 / math.sqrt(ff))
            st["gate_up_scales"] = st["down_scales"] = None
        else:
            st["gate_up"], st["gate_up_scales"] = _plain_quantize(normal(e, 2, ff, d) / math.sqrt(d), 128)
            st["down"], st["down_scales"] = _plain_quantize(normal(e, d, ff) / math.sqrt(ff), 128)
        st["residual"] = normal(n, d).to(_DT[case["x"]]) if case["residual"] else None
        st["y"] = torch.zeros(n, d, dtype=_DT[case["x"]], device="cuda")
        st["ids"] = torch.zeros(n, case["k"], dtype=torch.int32, device="cuda")
        st["weights"] = torch.zeros(n, case["k"], device="cuda")
    if own:
        from autoregressive_decode_step_gb300 import abi as A
        st["abi"] = A
        if case["op"] == "product":
            st["ws"] = A.workspace(A.ds_gemm_fp8_workspace_bytes(case["n"], case["rows"], case["cols"]))
        elif case["op"] == "experts":
            st["ws"] = A.workspace(A.ds_moe_layer_workspace_bytes(case["n"], case["d"], case["ff"], case["experts"],
                                                                  case["k"]))
    return st


# --------------------------------------------------------------------- run
def _own_quant(st):
    st["abi"].ds_fp8_quantize(st["x"], st["case"]["block"], st["q"], st["scales"])
    return dict(q=st["q"], scales=st["scales"])


def _plain_quant(st):
    q, scales = _plain_quantize(st["x"], st["case"]["block"])
    return dict(q=q, scales=scales)


def _own_product(st):
    st["abi"].ds_gemm_fp8(st["w"], st["w_scales"], st["x"], st["x_scales"], st["y"], st["ws"])
    return st["y"]


def _plain_product(st):
    y = _widen(st["x"], st["x_scales"], 1) @ _widen(st["w"], st["w_scales"], 128).t()
    return y.to(st["y"].dtype)


def _own_experts(st):
    c = st["case"]
    st["abi"].ds_moe_layer(st["x"], st["router"], c["k"], c["norm"], st["gate_up"], st["gate_up_scales"], st["down"],
                           st["down_scales"], st["residual"], st["y"], st["ids"], st["weights"], st["ws"])
    return dict(y=st["y"], ids=st["ids"], weights=st["weights"])


def _plain_experts(st):
    c = st["case"]
    n, d, ff, e, k = c["n"], c["d"], c["ff"], c["experts"], c["k"]
    # logits in 64 bits: two experts may be as close as that
    logits = st["x"].double() @ st["router"].double().t()
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.softmax(logits, 1).gather(1, ids)
    p = (p / p.sum(1, keepdim=True) if c["norm"] else p).float()
    x = st["x"].float()
    gate_up, down, gus, dns = st["gate_up"], st["down"], st["gate_up_scales"], st["down_scales"]
    few = n * k < e  # the chosen experts' matrices, or all experts' products with all tokens
    if few:
        at = ids.reshape(-1)
        if c["w"] == "e4m3":
            gate_up = gate_up.view(torch.uint8)[at].view(torch.float8_e4m3fn)
            down = down.view(torch.uint8)[at].view(torch.float8_e4m3fn)
            gus, dns = gus[at], dns[at]
        else:
            gate_up, down = gate_up[at], down[at]
        x = x.repeat_interleave(k, 0)[:, None]  # [pairs][1][d]
    gate_up = (gate_up.float() if gus is None else _widen(gate_up, gus, 128)).reshape(-1, 2 * ff, d)
    h = x @ gate_up.transpose(1, 2)  # [pairs][1][2 ff] or [experts][n][2 ff]
    del gate_up
    h = h[..., :ff] / (1 + torch.exp(-h[..., :ff])) * h[..., ff:]
    y = h @ (down.float() if dns is None else _widen(down, dns, 128)).transpose(1, 2)
    y = y.view(n, k, d) if few else y[ids, torch.arange(n, device="cuda")[:, None]]
    y = (y * p[..., None]).sum(1)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return dict(y=y.to(st["y"].dtype), ids=ids.to(torch.int32), weights=p)


def run(st):
    op = st["case"]["op"]
    if own:
        return _own_quant(st) if op == "quant" else _own_product(st) if op == "product" else _own_experts(st)
    return _plain_quant(st) if op == "quant" else _plain_product(st) if op == "product" else _plain_experts(st)


# -------------------------------------------------------------------- work
def _reached(case):
    """How many experts n tokens that choose k of them each reach (all being equally likely)."""
    e = case["experts"]
    return e * (1 - (1 - case["k"] / e) ** case["n"])


def work(case):
    if case["op"] == "quant":
        m = case["rows"] * case["cols"]
        scales = -(-case["rows"] // case["block"]) * -(-case["cols"] // 128)
        return {"bytes": m * (_SIZE[case["x"]] + 1) + 4 * scales, "flops": 2 * m}
    if case["op"] == "product":
        n, rows, cols = case["n"], case["rows"], case["cols"]
        kb = -(-cols // 128)
        return {"bytes": (n + rows) * cols + 4 * kb * (n + -(-rows // 128)) + n * rows * _SIZE[case["y"]],
                "flops": 2 * n * rows * cols}
    n, d, ff, e, k = case["n"], case["d"], case["ff"], case["experts"], case["k"]
    matrices = _reached(case) * 3 * d * ff * _SIZE[case["w"]] * (1 + 4 / 16384 if case["w"] == "e4m3" else 1)
    rows = n * d * _SIZE[case["x"]] * (3 if case["residual"] else 2)
    return {"bytes": matrices + rows + 2 * e * d + 8 * n * k, "flops": 2 * n * (e * d + k * 3 * d * ff)}


# ------------------------------------------------------------------- exact
def _e4m3(v):
    """The nearest number of sign, 4 bits of exponent and 3 of mantissa, ties to even, for |v| up to 464, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_quant(st):
    c = st["case"]
    x, br = st["x"].double(), c["block"]
    q = torch.empty(c["rows"], c["cols"], dtype=torch.float64, device="cuda")
    scales = torch.empty(st["scales"].shape, dtype=torch.float64, device="cuda")
    for j in range(scales.shape[1]):  # a column of blocks at a time
        part = x[:, 128 * j:128 * j + 128]
        rows = torch.nn.functional.pad(part.abs().amax(1), (0, -c["rows"] % br)).view(-1, br).amax(1)
        scales[:, j] = rows.clamp(min=TINY) / 448
        q[:, 128 * j:128 * j + 128] = _e4m3(part / scales[:, j].repeat_interleave(br)[:c["rows"], None])
    return dict(q=q, scales=scales)


def _exact_product(st):
    c = st["case"]
    y = torch.zeros(c["n"], c["rows"], dtype=torch.float64, device="cuda")
    of = torch.arange(c["rows"], device="cuda") // 128
    for b in range(-(-c["cols"] // 128)):
        part = st["x"][:, 128 * b:128 * b + 128].double() @ st["w"][:, 128 * b:128 * b + 128].double().t()
        y += part * st["x_scales"][:, b].double()[:, None] * st["w_scales"][of, b].double()
    return y


def _exact_matrix(w, scales):
    """One expert's matrix [rows][cols] in 64 bits."""
    m = w.double()
    if scales is not None:
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                m[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= scales[i, j].double()
    return m


def _exact_experts(st):
    c = st["case"]
    x = st["x"].double()
    score = torch.einsum("nd,ed->ne", x, st["router"].double()).cpu().numpy()
    ids = np.argsort(-score, axis=1, kind="stable")[:, :c["k"]]
    p = np.exp(score - score.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    p = np.take_along_axis(p, ids, 1)
    if c["norm"]:
        p /= p.sum(1, keepdims=True)
    y = torch.zeros_like(x) if st["residual"] is None else st["residual"].double()
    for e in np.unique(ids):
        token, slot = np.nonzero(ids == e)
        at = torch.from_numpy(token).cuda()
        gus = [None, None] if st["gate_up_scales"] is None else st["gate_up_scales"][e]
        gate = x[at] @ _exact_matrix(st["gate_up"][e, 0], gus[0]).t()
        up = x[at] @ _exact_matrix(st["gate_up"][e, 1], gus[1]).t()
        out = (gate * torch.sigmoid(gate) * up) @ _exact_matrix(
            st["down"][e], None if st["down_scales"] is None else st["down_scales"][e]).t()
        y.index_add_(0, at, out * torch.from_numpy(p[token, slot]).cuda()[:, None])
    return dict(y=y, ids=None, weights=torch.from_numpy(p))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    return _exact_quant(st) if op == "quant" else _exact_product(st) if op == "product" else _exact_experts(st)
