"""Measured calls of the ragged-batch operators over the paged K/V pool.

Three operators that a serving step of many requests runs in this order:

* ``plan``  block tables, row starts, positions and cache slots from the
  requests' lengths (``ds_paged_plan``);
* ``rope``  rotary positions of one or several axes for the rows of a fused
  q|k|v projection, k and v written to their cache slots
  (``ds_rope_append``);
* ``attn``  attention of every request's new rows (a chunk, or one token) over
  its blocks of the pool (``ds_gqa_chunk_attn``).

``run`` computes an operator in plain torch operations, or, with ``own`` true,
through the library.
"""
import math

import numpy as np
import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one user chatting: a single token over a 1,024-position context (the smallest call: latency)
        dict(name="attn token 1x1024", op="attn", kind="decode", seqs=1, new=1, lo=1024, hi=1024, nq=32, nkv=8, hd=128,
             bt=16, q="bf16", kv="bf16"),
        # a full decode batch, fp32 activations, contexts uniform in 128..4096
        dict(name="attn token 64x4096", op="attn", kind="decode", seqs=64, new=1, lo=128, hi=4096, nq=32, nkv=8, hd=128,
             bt=16, q="fp32", kv="bf16"),
        # one prompt chunk of 256 rows, fp32 activations, behind 768 cached positions
        dict(name="attn chunk 256@768", op="attn", kind="chunk", seqs=1, new=256, lo=1024, hi=1024, nq=32, nkv=8, hd=128,
             bt=16, q="fp32", kv="bf16"),
        # a mixed step: most requests decode, every ninth runs a chunk of up to 203 rows
        dict(name="attn mixed 28+4", op="attn", kind="mixed", seqs=32, new=203, lo=300, hi=4096, nq=32, nkv=8, hd=128,
             bt=16, q="bf16", kv="bf16"),
        # a whole long prompt at once (the largest call: tensor products)
        dict(name="attn prompt 8192", op="attn", kind="chunk", seqs=1, new=8192, lo=8192, hi=8192, nq=32, nkv=8, hd=128,
             bt=16, q="bf16", kv="bf16"),
        # ragged chunks of narrow heads in odd groups of seven, larger pages
        dict(name="attn ragged 7x64", op="attn", kind="ragged", seqs=5, new=333, lo=333, hi=2999, nq=14, nkv=2, hd=64,
             bt=32, q="bf16", kv="bf16"),
        # a short prompt of a model that keeps an fp32 cache
        dict(name="attn fp32 cache 512", op="attn", kind="chunk", seqs=1, new=512, lo=512, hi=512, nq=16, nkv=8, hd=128,
             bt=16, q="fp32", kv="fp32"),
        # the plan of a decode batch: one token a request
        dict(name="plan token 64", op="plan", kind="decode", seqs=64, new=1, hi=4096, bt=16, rows=64),
        # the plan of a step with many prompts: odd lengths, rows padded to a fixed count
        dict(name="plan prompts 16384", op="plan", kind="ragged", seqs=250, new=120, hi=4096, bt=16, rows=16384),
        # a decode batch's fused projection in fp32, one axis (text)
        dict(name="rope token 64", op="rope", rows=64, pad=0, axes=1, nq=32, nkv=8, hd=128, rot=128, layout=0, x="fp32",
             q="fp32", kv="bf16", maxpos=8192),
        # a prompt with video: three axes (time, height, width), bf16
        dict(name="rope video 8192", op="rope", rows=8192, pad=0, axes=3, nq=32, nkv=8, hd=128, rot=128, layout=0,
             x="bf16", q="bf16", kv="bf16", maxpos=8192),
        # an image's odd row count, interleaved pairs, part of each head rotated, far positions, padded rows, fp32 cache
        dict(name="rope image 1001", op="rope", rows=1001, pad=23, axes=3, nq=14, nkv=2, hd=80, rot=48, layout=1,
             x="fp32", q="fp32", kv="fp32", maxpos=1000000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "plan", "rope"])
    if op == "plan":
        return dict(op="plan", kind=rng.choice(["decode", "ragged"]), seqs=_log(rng, 1, 1000), new=_log(rng, 1, 120),
                    hi=_log(rng, 130, 8192), bt=rng.choice([8, 16, 32, 7]), rows=0)
    if op == "rope":
        hd = rng.choice([64, 80, 128])
        nkv = rng.choice([1, 2, 8])
        rows = _log(rng, 1, 8192)
        return dict(op="rope", rows=rows, pad=rng.choice([0, 0, 5]) if rows > 16 else 0, axes=rng.choice([1, 2, 3]),
                    nq=nkv * rng.choice([1, 2, 4]), nkv=nkv, hd=hd, rot=rng.choice([hd, hd // 2]),
                    layout=rng.choice([0, 1]), x=rng.choice(["fp32", "bf16"]), q=rng.choice(["fp32", "bf16"]),
                    kv=rng.choice(["fp32", "bf16"]), maxpos=_log(rng, 8192, 1000000))
    kind = rng.choice(["decode", "chunk", "mixed", "ragged"])
    nkv = rng.choice([1, 2, 4, 8])
    c = dict(op="attn", kind=kind, nq=nkv * rng.choice([1, 2, 3, 4, 7]), nkv=nkv, hd=rng.choice([64, 128, 128]),
             bt=rng.choice([8, 16, 16, 32, 64]), q=rng.choice(["bf16", "bf16", "fp32"]), kv="bf16")
    if kind == "decode":
        c.update(seqs=_log(rng, 1, 64), new=1, lo=1, hi=_log(rng, 64, 4096))
    elif kind == "chunk":
        c.update(seqs=1, new=_log(rng, 2, 3001))
        c["lo"] = c["hi"] = c["new"] + _log(rng, 1, 4096)
    else:
        c.update(seqs=rng.randrange(2, 21), new=_log(rng, 8, 300))
        c.update(lo=c["new"], hi=c["new"] + _log(rng, 16, 3500))
    if rng.random() < 0.15:  # a model that keeps an fp32 cache
        c.update(q="fp32", kv="fp32")
    return c


def _lengths(case):
    """(new rows, total length) of every request: whole numbers that follow from the case's sizes alone."""
    g = np.random.RandomState(case["seqs"] * 7919 + case["new"] * 31 + case["hi"])
    n, new = case["seqs"], case["new"]
    if case["op"] == "plan":
        rows = np.ones(n, np.int64) if case["kind"] == "decode" else g.randint(0, new + 1, n)
        return rows, rows + g.randint(0, max(1, case["hi"] - new), n)
    if case["kind"] == "decode":
        rows = np.ones(n, np.int64)
    elif case["kind"] == "chunk":
        rows = np.full(n, new)
    elif case["kind"] == "mixed":
        rows = np.where(np.arange(n) % 9 == 4, g.randint(new // 2, new + 1, n), 1)
    else:
        rows = g.randint(1, new + 1, n)
    return rows, np.maximum(rows, g.randint(case["lo"], case["hi"] + 1, n))


def _pair_axes(case):
    """The axis of every rotated pair: the first quarter turns by time, the rest alternates height and width in two runs."""
    half, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return np.zeros(half, np.uint8)
    cuts = [half // 4 + (half - half // 4) * a // (axes - 1) for a in range(axes - 1)]
    return np.searchsorted(np.array(cuts), np.arange(half), side="right").astype(np.uint8)


BASE = 500000.0


# ----------------------------------------------------------------- prepare
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rs = np.random.RandomState(seed)
    st = {"case": case}

    def i32(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    if case["op"] == "plan":
        new, total = _lengths(case)
        bt, n = case["bt"], case["seqs"]
        cached = total - new
        new, cached = rs.permutation(new), rs.permutation(cached)
        had = -(-cached // bt)
        need = -(-(cached + new) // bt) - had
        width = -(-(int(cached.max()) + int(new.max())) // bt) + 2
        blocks = int((had + need).sum()) + 100
        order = rs.permutation(blocks)
        table = np.full((n, width), -1, np.int64)
        at = 0
        for s in range(n):
            table[s, :had[s]] = order[at:at + had[s]]
            at += had[s]
        rows = max(case["rows"] or int(new.sum()), 1)
        st.update(cached=i32(cached), new=i32(new), free=i32(order[at:]), table=i32(table), rows=rows,
                  cache_rows=blocks * bt, width=table.shape[1])
        if rows < new.sum():
            raise ValueError("rows do not fit")
        # the buffers that a serving loop keeps from step to step
        st["out"] = {k: torch.zeros(m, dtype=torch.int32, device="cuda") for k, m in
                     (("row_starts", n + 1), ("seq_lens", n), ("row_seq", rows), ("positions", rows), ("slots", rows),
                      ("n_taken", 1))}
        nbytes = 256
    elif case["op"] == "rope":
        rows, nq, nkv, hd = case["rows"], case["nq"], case["nkv"], case["hd"]
        st["x"] = normal(rows, (nq + 2 * nkv) * hd).to(_DT[case["x"]])
        st["pos"] = torch.randint(0, case["maxpos"], (case["axes"], rows), generator=g, device="cuda", dtype=torch.int32)
        cache_rows = rows + 16
        slots = rs.permutation(cache_rows)[:rows]
        if case["pad"]:  # the last rows of a padded batch belong to no request
            slots[max(0, rows - case["pad"]):] = -1
        st["slots"] = i32(slots)
        st["k"] = torch.zeros(cache_rows, nkv * hd, dtype=_DT[case["kv"]], device="cuda")
        st["v"] = torch.zeros(cache_rows, nkv * hd, dtype=_DT[case["kv"]], device="cuda")
        st["q"] = torch.zeros(rows, nq * hd, dtype=_DT[case["q"]], device="cuda")
        st["axes"] = _pair_axes(case)
        nbytes = 256
    else:
        new, total = _lengths(case)
        bt, n, nq, nkv, hd = case["bt"], case["seqs"], case["nq"], case["nkv"], case["hd"]
        had = -(-total // bt)
        width, blocks = int(had.max()), int(had.sum()) + 3
        order = rs.permutation(blocks)
        table = np.zeros((n, width), np.int64)
        at = 0
        for s in range(n):
            table[s, :had[s]] = order[at:at + had[s]]
            at += had[s]
        rows = int(new.sum())
        starts = np.concatenate([[0], np.cumsum(new)])
        st.update(rows=rows, width=width, cache_rows=blocks * bt, max_new=int(new.max()), max_len=int(total.max()),
                  starts=i32(starts), lens=i32(total), table=i32(table), host_new=new, host_len=total,
                  scale=1.0 / math.sqrt(hd))
        st["q"] = normal(rows, nq * hd).to(_DT[case["q"]])
        st["k"] = normal(blocks * bt, nkv * hd, dtype=_DT[case["kv"]])
        st["v"] = normal(blocks * bt, nkv * hd, dtype=_DT[case["kv"]])
        st["out"] = torch.zeros_like(st["q"])
        nbytes = 0
    if own:
        from autoregressive_decode_step_gb300 import abi as A
        st["abi"] = A
        st["ws"] = A.workspace(nbytes or A.ds_chunk_attention_workspace_bytes(case["seqs"], st["rows"], case["nq"],
                                                                              case["nkv"], case["hd"]))
    return st


# --------------------------------------------------------------------- run
def _own_plan(st):
    c, o = st["case"], st["out"]
    st["abi"].ds_paged_plan(st["cached"], st["new"], c["seqs"], st["free"], c["bt"], st["cache_rows"], st["table"],
                            st["width"], o["row_starts"], o["seq_lens"], o["row_seq"], o["positions"], o["slots"],
                            st["rows"], o["n_taken"], st["ws"])
    return dict(o, block_table=st["table"])


def _plain_plan(st):
    c, bt, rows, free, table = st["case"], st["case"]["bt"], st["rows"], st["free"], st["table"]
    cached, new = st["cached"].long(), st["new"].long()
    total = cached + new
    had = (cached + bt - 1) // bt
    need = (total + bt - 1) // bt - had
    row_end, blk_end = torch.cumsum(new, 0), torch.cumsum(need, 0)
    first = torch.cat([torch.zeros_like(row_end[:1]), row_end])
    r = torch.arange(rows, device="cuda")
    s = torch.searchsorted(row_end, r, right=True)
    live = s < c["seqs"]
    s = s.clamp(max=c["seqs"] - 1)
    pos = cached[s] + r - first[s]
    col = torch.arange(st["width"], device="cuda")[None, :]
    took = (blk_end - need)[:, None] + col - had[:, None]
    fresh = (col >= had[:, None]) & (col < (had + need)[:, None])
    table.copy_(torch.where(fresh, free[took.clamp(0, free.numel() - 1)], table))
    slot = table[s, (pos // bt).clamp(max=st["width"] - 1)].long() * bt + pos % bt
    minus = torch.full_like(r, -1)

    def i32(v):
        return v.to(torch.int32)

    return dict(row_starts=i32(first), seq_lens=i32(total), row_seq=i32(torch.where(live, s, minus)),
                positions=i32(torch.where(live, pos, minus)), slots=i32(torch.where(live, slot, minus)),
                n_taken=i32(blk_end[-1:]), block_table=table)


def _own_rope(st):
    c = st["case"]
    st["abi"].ds_rope_append(st["x"], st["x"].shape[1], c["rows"], st["pos"], c["axes"], st["axes"], c["nq"], c["nkv"],
                             c["hd"], c["rot"], BASE, c["layout"], st["q"], st["k"], st["v"], st["k"].shape[0],
                             st["slots"], st["ws"])
    return st["q"], st["k"], st["v"]


def _rotate(x, cos, sin, case):
    """x [rows][heads][hd] with the first rot dims of every head turned; cos and sin [rows][1][rot / 2]."""
    rot = case["rot"]
    if case["layout"] == 0:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def _plain_rope(st):
    c = st["case"]
    rows, nq, nkv, hd, rot = c["rows"], c["nq"], c["nkv"], c["hd"], c["rot"]
    pair = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    axis = torch.from_numpy(st["axes"]).to("cuda", torch.int64)
    angle = st["pos"].t()[:, axis].double() * BASE ** (-2.0 * pair / rot)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = st["x"].float().view(rows, nq + 2 * nkv, hd)
    y = _rotate(x[:, :nq + nkv], cos, sin, c)
    live = st["slots"] >= 0
    # rows of padding leave q as it was, and write the first row's k and v once more (it is never padding)
    st["q"].copy_(torch.where(live[:, None], y[:, :nq].reshape(rows, -1).to(st["q"].dtype), st["q"]))
    slot, k, v = st["slots"].long(), y[:, nq:], x[:, nq + nkv:]
    if c["pad"]:
        slot = torch.where(live, slot, slot[:1])
        k, v = torch.where(live[:, None, None], k, k[:1]), torch.where(live[:, None, None], v, v[:1])
    st["k"].index_copy_(0, slot, k.reshape(rows, nkv * hd).to(st["k"].dtype))
    st["v"].index_copy_(0, slot, v.reshape(rows, nkv * hd).to(st["v"].dtype))
    return st["q"], st["k"], st["v"]


def _own_attn(st):
    c = st["case"]
    st["abi"].ds_gqa_chunk_attn(st["q"], st["rows"], st["starts"], st["lens"], c["seqs"], st["k"], st["v"],
                                st["cache_rows"], st["table"], st["width"], c["bt"], c["nq"], c["nkv"], c["hd"],
                                st["scale"], st["out"], st["ws"])
    return st["out"]


def _plain_attn(st):
    c = st["case"]
    n, m, L, nq, nkv, hd, bt = c["seqs"], st["max_new"], st["max_len"], c["nq"], c["nkv"], c["hd"], c["bt"]
    starts, lens = st["starts"].long(), st["lens"].long()
    new = starts[1:] - starts[:-1]
    # every request padded to the longest: its keys and values gathered from its blocks, its rows from the batch
    t = torch.arange(L, device="cuda")
    slot = st["table"].long()[:, t // bt] * bt + t % bt
    k = st["k"][slot].float().view(n, L, nkv, hd).permute(0, 2, 3, 1)
    v = st["v"][slot].float().view(n, L, nkv, hd).permute(0, 2, 1, 3)
    j = torch.arange(m, device="cuda")
    row = (starts[:-1, None] + j).clamp(max=st["rows"] - 1)
    q = st["q"][row].float().view(n, m, nkv, nq // nkv, hd).permute(0, 2, 3, 1, 4).reshape(n, nkv, -1, hd)
    score = (q @ k).mul_(st["scale"]).view(n, nkv, nq // nkv, m, L)
    hidden = t[None, None, :] > (lens - new)[:, None, None] + j[None, :, None]
    score.masked_fill_(hidden[:, None, None], float("-inf"))
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score.view(n, nkv, -1, L) @ v).view(n, nkv, nq // nkv, m, hd) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(n, m, nq * hd)
    r = torch.arange(st["rows"], device="cuda")
    s = torch.searchsorted(starts[1:], r, right=True)
    return out[s, r - starts[s]].to(st["q"].dtype)


def run(st):
    op = st["case"]["op"]
    if own:
        return _own_plan(st) if op == "plan" else _own_rope(st) if op == "rope" else _own_attn(st)
    return _plain_plan(st) if op == "plan" else _plain_rope(st) if op == "rope" else _plain_attn(st)


# -------------------------------------------------------------------- work
def work(case):
    size = {"fp32": 4, "bf16": 2}
    if case["op"] == "plan":
        new, total = _lengths(case)
        bt, n = case["bt"], case["seqs"]
        # the seed's permutation changes which request needs a block, hardly how many
        taken = int((-(-total // bt) + -(-(total - new) // bt) * -1).sum())
        rows = max(case["rows"] or int(new.sum()), 1)
        return {"bytes": 16 * n + 12 * rows + 8 * taken, "flops": 0}
    if case["op"] == "rope":
        live = max(case["rows"] - case["pad"], 0)
        e = case["hd"]
        nbytes = live * ((case["nq"] + 2 * case["nkv"]) * e * size[case["x"]] + 4 * case["axes"]
                         + case["nq"] * e * size[case["q"]] + 2 * case["nkv"] * e * size[case["kv"]]) + 4 * case["rows"]
        return {"bytes": nbytes, "flops": 3 * live * (case["nq"] + case["nkv"]) * case["rot"]}
    new, total = _lengths(case)
    attended = int((new * (total - new) + new * (new + 1) // 2).sum())
    io = 2 * int(new.sum()) * case["nq"] * case["hd"] * size[case["q"]]
    kv = 2 * int(total.sum()) * case["nkv"] * case["hd"] * size[case["kv"]]
    return {"bytes": io + kv, "flops": 4 * case["hd"] * case["nq"] * attended}


# ------------------------------------------------------------------- exact
def _exact_rope(st):
    c = st["case"]
    nq, nkv, hd, rot = c["nq"], c["nkv"], c["hd"], c["rot"]
    x = st["x"].double().cpu().numpy().reshape(c["rows"], nq + 2 * nkv, hd)
    pos, slots = st["pos"].cpu().numpy().astype(np.float64), st["slots"].cpu().numpy()
    out = x.copy()
    for p in range(rot // 2):  # one pair of every head at a time
        a = pos[st["axes"][p]] * np.exp(-2.0 * p / rot * np.log(BASE))
        i, j = (p, p + rot // 2) if c["layout"] == 0 else (2 * p, 2 * p + 1)
        turned = (x[:, :nq + nkv, i] + 1j * x[:, :nq + nkv, j]) * np.exp(1j * a)[:, None]
        out[:, :nq + nkv, i], out[:, :nq + nkv, j] = turned.real, turned.imag
    q = np.zeros((c["rows"], nq * hd))
    k = np.zeros((st["k"].shape[0], nkv * hd))
    v = np.zeros_like(k)
    live = slots >= 0
    q[live] = out[live, :nq].reshape(-1, nq * hd)
    k[slots[live]] = out[live, nq:nq + nkv].reshape(-1, nkv * hd)
    v[slots[live]] = out[live, nq + nkv:].reshape(-1, nkv * hd)
    return tuple(torch.from_numpy(a) for a in (q, k, v))


def _exact_attn(st):
    c = st["case"]
    nq, nkv, hd, bt = c["nq"], c["nkv"], c["hd"], c["bt"]
    out = torch.empty(st["rows"], nq, hd, dtype=torch.float64, device="cuda")
    table, at = st["table"].cpu().numpy(), 0
    q = st["q"].view(st["rows"], nq, hd)
    for s in range(c["seqs"]):
        m, L = int(st["host_new"][s]), int(st["host_len"][s])
        rows = (table[s][:, None].astype(np.int64) * bt + np.arange(bt)).reshape(-1)[:L]
        rows = torch.from_numpy(rows).cuda()
        for h in range(nkv):
            k = st["k"][rows, h * hd:(h + 1) * hd].double()
            v = st["v"][rows, h * hd:(h + 1) * hd].double()
            for i in range(nq // nkv):
                head = h * (nq // nkv) + i
                for a in range(0, m, 2048):  # so many rows at a time
                    b = min(m, a + 2048)
                    seen = L - m + b
                    e = torch.einsum("id,td->it", q[at + a:at + b, head].double(), k[:seen]) * st["scale"]
                    last = L - m + torch.arange(a, b, device="cuda")
                    e[torch.arange(seen, device="cuda")[None, :] > last[:, None]] = -math.inf
                    w = torch.softmax(e, dim=1)
                    out[at + a:at + b, head] = torch.einsum("it,td->id", w, v[:seen])
        at += m
    return out.view(st["rows"], nq * hd)


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    st = prepare(case, seed)
    return _exact_rope(st) if case["op"] == "rope" else _exact_attn(st)
