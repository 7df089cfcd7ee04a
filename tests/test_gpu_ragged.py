"""The ragged-step operators on the GPU against plain 64-bit statements:
ds_paged_plan (whole numbers, exact), ds_rope_append, ds_gqa_chunk_attn, and
the three run together as a serving loop uses them.

Tolerances come from the roundings on the way (u = 2^-24 for fp32, h = 2^-8
for bf16, half a step relative to the value each):
* a rotated value x cos - y sin: sine and cosine within 4u (argument and
  function), two products and one sum: |error| <= 8u (|x| + |y|), then the
  output type's rounding of the value;
* attention: a score is a sum of hd products, off by at most
  d = (hd + 4) u scale sum|q_i k_i|, so each weight by a factor e^(+-2d) at
  most (its own score and the sum's); the sum over T positions adds (T + 8) u;
  a bf16 kernel also rounds each weight (h).  So
  |error| <= (2d + (T + 8) u [+ h]) max|v| + rounding of the output.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from autoregressive_decode_step_gb300 import abi
    return abi


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


# ------------------------------------------------------------------- plan
def plan_reference(cached, new, free, bt, pool_blocks, table, max_rows):
    """The plan, one sequence and one row at a time."""
    n, width = table.shape
    table = table.copy()
    starts, lens, taken, err = [0], [], 0, 0
    row_seq, pos, slots = [-1] * max_rows, [-1] * max_rows, [-1] * max_rows
    ended = False
    for s in range(n):
        c, m = int(cached[s]), int(new[s])
        if c < 0 or m < 0 or c + m > width * bt:
            err |= 2
            m, had, need = 0, 0, 0
        else:
            had = -(-c // bt)
            need = -(-(c + m) // bt) - had
        if not ended and (starts[-1] + m > max_rows or taken + need > len(free)):
            ended = True
            err |= 16
        if ended:
            m = need = 0
        for i in range(need):
            b = int(free[taken + i])
            if b < 0 or b >= pool_blocks:
                err |= 2
                b = -1
            table[s, had + i] = b
        for j in range(m):
            r = starts[-1] + j
            row_seq[r], pos[r] = s, c + j
            b = int(table[s, (c + j) // bt])
            if b < 0 or b >= pool_blocks:
                err |= 2
            else:
                slots[r] = b * bt + (c + j) % bt
        starts.append(starts[-1] + m)
        taken += need
        lens.append(min(max(c, 0), width * bt) + m)
    return dict(row_starts=starts, seq_lens=lens, row_seq=row_seq, positions=pos, slots=slots, n_taken=[taken],
                block_table=table, err=err)


def run_plan(A, cached, new, free, bt, cache_rows, table, max_rows, stream=None):
    n, width = table.shape
    out = {k: torch.full((m,), -77, dtype=torch.int32, device="cuda") for k, m in
           (("row_starts", n + 1), ("seq_lens", n), ("row_seq", max_rows), ("positions", max_rows),
            ("slots", max_rows), ("n_taken", 1))}
    t = i32(table)
    ws = A.workspace(A.ds_paged_plan_workspace_bytes())
    args = (i32(cached), i32(new), n, i32(free) if len(free) else None, bt, cache_rows, t, width, out["row_starts"],
            out["seq_lens"], out["row_seq"], out["positions"], out["slots"], max_rows, out["n_taken"], ws)
    A.ds_paged_plan(*args, stream=stream)
    first = {k: v.clone() for k, v in out.items()}
    A.ds_paged_plan(*args, stream=stream)  # the lengths stay, so the same call gives the same answer
    for k in out:
        assert torch.equal(first[k], out[k]), k
    return dict(out, block_table=t, err=A.ds_workspace_error(ws))


def check_plan(got, want):
    assert got["err"] == want["err"]
    for k in want:
        if k != "err":
            assert got[k].cpu().numpy().tolist() == np.asarray(want[k]).tolist(), k


@pytest.mark.parametrize("n,bt,hi_new,hi_cached,pad", [
    (1, 16, 1, 0, 0), (1, 16, 40, 100, 3), (64, 16, 1, 4096, 0), (250, 16, 60, 300, 11), (257, 7, 9, 40, 0),
    (1000, 1, 5, 9, 1), (4096, 32, 3, 100, 0), (33, 128, 300, 500, 200),
])
def test_plan_matches_the_plain_statement(A, n, bt, hi_new, hi_cached, pad):
    g = np.random.RandomState(n * 7 + bt)
    new = g.randint(0, hi_new + 1, n)
    new[-1] = hi_new
    cached = g.randint(0, hi_cached + 1, n)
    had = -(-cached // bt)
    need = -(-(cached + new) // bt) - had
    blocks = int((had + need).sum()) + 5
    order = g.permutation(blocks)
    table = np.full((n, int((had + need).max()) + 1), -5)
    at = 0
    for s in range(n):
        table[s, :had[s]] = order[at:at + had[s]]
        at += had[s]
    rows = int(new.sum()) + pad
    want = plan_reference(cached, new, order[at:], bt, blocks, table, rows)
    assert want["err"] == 0
    check_plan(run_plan(A, cached, new, order[at:], bt, blocks * bt, table, rows), want)


@pytest.mark.parametrize("case", ["no free list", "blocks run out", "rows run out", "bad lengths", "bad blocks",
                                  "empty step"])
def test_plan_limits(A, case):
    bt, width, blocks = 4, 6, 64
    cached = np.array([5, 0, 8, 3, 24, 7])
    new = np.array([3, 6, 0, 2, 0, 9])
    table = np.arange(36).reshape(6, 6) % blocks
    free, rows = np.arange(40, 60), 32
    if case == "no free list":
        free = free[:0]
    elif case == "blocks run out":
        free = free[:3]
    elif case == "rows run out":
        rows = 10
    elif case == "bad lengths":
        cached[1], new[3], cached[5] = -3, -1, 20
    elif case == "bad blocks":
        free = free.copy()
        free[0], free[2] = 64, -9
        table[3, 0] = 99
    else:
        new[:] = 0
    want = plan_reference(cached, new, free, bt, blocks, table, rows)
    check_plan(run_plan(A, cached, new, free, bt, blocks * bt, table, rows), want)


# ------------------------------------------------------------------- rope
def rope_reference(x, pos, pair_axis, nq, nkv, hd, rot, base, layout):
    """fp64: (rotated q, rotated k, v) and the magnitude |x| + |y| behind every element."""
    x = x.double().cpu().numpy().reshape(x.shape[0], nq + 2 * nkv, hd)
    y, mag = x.copy(), np.zeros_like(x)
    for p in range(rot // 2):
        a = pos[pair_axis[p]].astype(np.float64) * float(base) ** (-2.0 * p / rot)
        i, j = (p, p + rot // 2) if layout == 0 else (2 * p, 2 * p + 1)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        u, v = x[:, :nq + nkv, i], x[:, :nq + nkv, j]
        y[:, :nq + nkv, i], y[:, :nq + nkv, j] = u * c - v * s, v * c + u * s
        mag[:, :nq + nkv, i] = mag[:, :nq + nkv, j] = abs(u) + abs(v)
    return y, mag


def near(got, want, mag):
    half = U if got.dtype == F32 else H
    g = got.double().cpu().numpy()
    slack = 8 * U * mag
    bad = np.abs(g - want) > slack + half * (np.abs(want) + slack)
    assert not bad.any(), (int(bad.sum()), float(np.abs(g - want).max()))


@pytest.mark.parametrize("rows,nq,nkv,hd,rot,layout,axes,xt,qt,kt,extra", [
    (1, 32, 8, 128, 128, 0, 1, F32, F32, BF16, 0),
    (64, 32, 8, 128, 128, 0, 1, F32, BF16, BF16, 0),
    (37, 14, 2, 64, 64, 0, 3, BF16, BF16, BF16, 8),
    (37, 14, 2, 64, 64, 1, 3, BF16, F32, F32, 16),
    (19, 4, 4, 80, 48, 1, 2, F32, F32, F32, 0),
    (19, 3, 1, 80, 40, 0, 3, BF16, BF16, F32, 0),      # rot no multiple of 16: single elements
    (7, 4, 2, 4, 4, 1, 1, F32, F32, F32, 0),           # the tiny decoder's heads
    (5, 2, 1, 6, 2, 0, 2, F32, F32, BF16, 3),          # odd strides
    (9, 2, 2, 256, 256, 0, 3, BF16, BF16, BF16, 0),
    (300, 8, 1, 128, 64, 0, 8, BF16, F32, BF16, 24),
    (2100, 4, 2, 64, 64, 0, 3, BF16, BF16, BF16, 8),   # many rows: the shared-memory ring
    (2500, 5, 1, 128, 96, 1, 2, F32, BF16, F32, 0),
    (4001, 1, 1, 16, 16, 0, 1, F32, F32, BF16, 0),
    (2048, 2, 1, 40, 24, 0, 1, BF16, F32, BF16, 0),    # many rows of single elements
])
@pytest.mark.parametrize("maxpos", [64, 2 ** 31 - 1])
def test_rope_append_matches_fp64(A, rows, nq, nkv, hd, rot, layout, axes, xt, qt, kt, extra, maxpos):
    g = torch.Generator().manual_seed(rows * 31 + hd + axes)
    cols, base = (nq + 2 * nkv) * hd, 500000.0
    wide = torch.randn(rows, cols + extra, generator=g).to(xt).cuda()
    pos = torch.randint(0, maxpos, (axes, rows), generator=g, dtype=torch.int64).to(torch.int32)
    pos[:, 0] = 0 if maxpos == 64 else maxpos
    pair_axis = np.random.RandomState(rows).randint(0, axes, rot // 2).astype(np.uint8)
    cache_rows = rows + 9
    slots = torch.randperm(cache_rows, generator=g)[:rows].to(torch.int32)
    if rows > 4:
        slots[rows // 2] = -1  # padding in the middle, and at the end
        slots[-1] = -1
    marks = [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in
             (((rows, nq * hd), qt), ((cache_rows, nkv * hd), kt), ((cache_rows, nkv * hd), kt))]
    q, k, v = marks
    ws = A.workspace(A.ds_rope_append_workspace_bytes())
    A.ds_rope_append(wide, cols + extra, rows, pos.cuda(), axes, None if axes == 1 else pair_axis, nq, nkv, hd, rot,
                     base, layout, q, k, v, cache_rows, slots.cuda(), ws)
    want, mag = rope_reference(wide[:, :cols], pos.numpy(), pair_axis, nq, nkv, hd, rot, base, layout)
    live = (slots >= 0).numpy()
    near(q[torch.from_numpy(live).cuda()], want[live, :nq].reshape(-1, nq * hd), mag[live, :nq].reshape(-1, nq * hd))
    at = slots[torch.from_numpy(live)].long().cuda()
    near(k[at], want[live, nq:nq + nkv].reshape(-1, nkv * hd), mag[live, nq:nq + nkv].reshape(-1, nkv * hd))
    near(v[at], want[live, nq + nkv:].reshape(-1, nkv * hd), mag[live, nq + nkv:].reshape(-1, nkv * hd))
    # what belongs to no row stays
    assert (q[torch.from_numpy(~live).cuda()] == 7).all()
    rest = torch.ones(cache_rows, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (k[rest] == 7).all() and (v[rest] == 7).all()
    assert A.ds_workspace_error(ws) == 0


def test_rope_append_with_one_axis_is_the_token_rotation(A):
    """The same angles as ds_rope's to their roundings: 8u (|x| + |y|) on either side."""
    x = torch.randn(1, (32 + 16) * 128, device="cuda")
    pos = i32([[4097]])
    q, k = torch.zeros(1, 32 * 128, device="cuda"), torch.zeros(1, 8 * 128, device="cuda")
    v, ws = torch.zeros_like(k), A.workspace(256)
    A.ds_rope_append(x, x.shape[1], 1, pos, 1, None, 32, 8, 128, 128, 10000.0, 0, q, k, v, 1, i32([0]), ws)
    q1, k1 = x[0, :4096].clone(), x[0, 4096:5120].clone()
    A.ds_rope(q1, k1, 4097, 32, 8, 128, 10000.0, 0)
    bound = 16 * U * 2 * float(x.abs().max())
    assert (q[0] - q1).abs().max() <= bound and (k[0] - k1).abs().max() <= bound
    assert torch.equal(v[0], x[0, 5120:])


def test_rope_append_with_all_buffers_in_one(A):
    """The rows first, their outputs behind them in the same storage."""
    rows = 5
    buf = torch.randn(rows * (6 + 2) * 64 + 2 * 8 * 128, device="cuda")
    x, rest = buf[:rows * 6 * 64].view(rows, 6 * 64), buf[rows * 6 * 64:]
    q, k, v = rest[:rows * 128].view(rows, 128), rest[rows * 128:][:8 * 128].view(8, 128), rest[-8 * 128:].view(8, 128)
    want, ws, args = [torch.zeros_like(t) for t in (q, k, v)], A.workspace(256), (i32([range(rows)]), 1, None, 2, 2, 64, 64, 1e4, 0)
    A.ds_rope_append(x, 6 * 64, rows, *args, q, k, v, 8, i32(range(rows)), ws)
    A.ds_rope_append(x.clone(), 6 * 64, rows, *args, *want, 8, i32(range(rows)), ws)
    assert torch.equal(q, want[0]) and torch.equal(k[:rows], want[1][:rows]) and torch.equal(v[:rows], want[2][:rows])


def test_rope_append_flags_and_skips_bad_rows_among_many(A):
    n = 3000
    x = torch.randn(n, 6 * 64, device="cuda")
    x[5] = float("nan")  # padding may hold anything
    pos, slots = torch.arange(n, dtype=torch.int32), torch.arange(n, dtype=torch.int32)
    slots[5], slots[700], pos[2999] = -1, n, -4
    q, k = torch.full((n, 128), 7.0, device="cuda"), torch.full((n, 128), 7.0, device="cuda")
    v, ws = k.clone(), A.workspace(256)
    A.ds_rope_append(x, 6 * 64, n, pos.cuda(), 1, None, 2, 2, 64, 64, 1e4, 0, q, k, v, n, slots.cuda(), ws)
    assert A.ds_workspace_error(ws) == A.DS_ERR_POSITION
    out = [5, 700, 2999]
    rest = torch.ones(n, dtype=torch.bool)
    rest[out] = False
    rest = rest.cuda()
    assert (q[out] == 7).all() and (k[out] == 7).all() and (v[out] == 7).all()
    assert torch.equal(v[rest], x[rest, 256:]) and not (q[rest] == 7).any()


def test_rope_append_flags_and_skips_bad_rows(A):
    x = torch.randn(4, 6 * 64, device="cuda")
    q, k = torch.full((4, 128), 7.0, device="cuda"), torch.full((8, 128), 7.0, device="cuda")
    v, ws = k.clone(), A.workspace(256)
    A.ds_rope_append(x, 6 * 64, 4, i32([[3, 1, -1, 5]]), 1, None, 2, 2, 64, 64, 1e4, 0, q, k, v, 8, i32([2, 8, 4, 5]),
                     ws)
    assert A.ds_workspace_error(ws) == A.DS_ERR_POSITION
    assert (q[1] == 7).all() and (q[2] == 7).all() and (k[4] == 7).all() and (v[4] == 7).all()
    assert torch.equal(v[2], x[0, 256:]) and torch.equal(v[5], x[3, 256:])


# -------------------------------------------------------------- attention
def pool(new, total, bt, nkv, hd, kvt, seed, paged=True, fill=None):
    """A pool with every sequence's blocks scattered in it: (k, v, table, width, cache_rows)."""
    g = torch.Generator().manual_seed(seed)
    had = [max(1, -(-t // bt)) for t in total]
    width = max(had) + 1
    blocks = len(total) * width + 3
    rows = blocks * bt
    k = torch.randn(rows, nkv * hd, generator=g).to(kvt)
    v = torch.randn(rows, nkv * hd, generator=g).to(kvt)
    if paged:
        order = torch.randperm(blocks, generator=g)[:len(total) * width].view(len(total), width)
    else:
        order = torch.arange(len(total) * width).view(len(total), width)
    return k, v, order.to(torch.int32), width, rows


def slots_of(table, s, length, bt):
    t = torch.arange(length)
    return table[s].long()[t // bt] * bt + t % bt


def attn_reference(q, k, v, table, starts, total, bt, nq, nkv, hd, scale):
    """fp64, sequence by sequence: outputs and the bound's d and max|v| per row."""
    out = torch.zeros(q.shape[0], nq, hd, dtype=torch.float64)
    d = torch.zeros(q.shape[0], nq, 1, dtype=torch.float64)
    vmax = torch.zeros_like(d)
    G = nq // nkv
    qd = q.double().view(-1, nq, hd)
    for s in range(len(total)):
        at = slots_of(table, s, total[s], bt)
        ks, vs = k[at].double().view(-1, nkv, hd), v[at].double().view(-1, nkv, hd)
        n = starts[s + 1] - starts[s]
        for j in range(n):
            seen = total[s] - n + j + 1
            if seen <= 0:
                continue
            r = starts[s] + j
            kk = ks[:seen].repeat_interleave(G, 1)
            vv = vs[:seen].repeat_interleave(G, 1)
            e = torch.einsum("hd,thd->ht", qd[r], kk) * scale
            w = torch.softmax(e, 1)
            out[r] = torch.einsum("ht,thd->hd", w, vv)
            d[r] = ((hd + 4) * U * scale * torch.einsum("hd,thd->ht", qd[r].abs(), kk.abs()).amax(1))[:, None]
            vmax[r] = vv.abs().amax((0, 2))[:, None]
    return out.view(q.shape[0], -1), d, vmax


def run_attn(A, q, k, v, table, starts, total, bt, nq, nkv, hd, scale, width, paged=True, n_rows=None, ws=None,
             stream=None):
    n_rows = n_rows or q.shape[0]
    ws = A.workspace(A.ds_chunk_attention_workspace_bytes(len(total), n_rows, nq, nkv, hd)) if ws is None else ws
    out = torch.full_like(q, 7.0, device="cuda")
    A.ds_gqa_chunk_attn(q.cuda(), n_rows, i32(starts), i32(total), len(total), k.cuda(), v.cuda(), k.shape[0],
                        table.cuda() if paged else None, width, bt, nq, nkv, hd, scale, out, ws, stream=stream)
    return out, ws


def attn_near(got, want, d, vmax, T, nq, hd, rounded_weights):
    half = U if got.dtype == F32 else H
    slack = ((2 * d + (T + 8) * U + (H if rounded_weights else 0)) * vmax).expand(-1, nq, hd).reshape(got.shape[0], -1)
    err = (got.double().cpu() - want).abs()
    bad = err > slack + half * (want.abs() + slack)
    assert not bad.any(), (int(bad.sum()), float(err.max()))


SHAPES = [
    # new rows, total lengths, bt, nq, nkv, hd
    ([1], [1], 16, 4, 2, 4),                           # the smallest: the tiny decoder's heads
    ([1], [1024], 16, 32, 8, 128),                     # a single token, split over CTAs
    ([1, 1, 1, 1], [1, 17, 300, 129], 16, 32, 8, 128),  # a decode batch
    ([130], [130], 16, 8, 2, 128),                     # a prompt from position 0
    ([70], [333], 16, 14, 2, 64),                      # a chunk behind a context, groups of seven
    ([1, 65, 0, 7, 1], [900, 65, 40, 511, 64], 16, 16, 8, 128),  # mixed, one sequence without rows
    ([33, 5], [140, 5], 32, 6, 2, 64),                 # groups of three
    ([9, 20], [30, 21], 5, 4, 4, 64),                  # odd pages
    ([40], [200], 1, 8, 1, 128),                       # pages of one position
    ([12], [77], 16, 3, 1, 80),                        # heads of 80
    ([10], [90], 8, 4, 1, 256),                        # heads of 256
    ([6], [150], 64, 150, 1, 64),                      # 150 heads share one
    ([300], [1300], 128, 4, 1, 128),
    ([3, 4], [2, 4], 16, 8, 2, 128),                   # a row that attends nothing
    ([2, 3, 150], [0, 3, 20], 16, 4, 2, 64),           # a sequence of length zero, most of a chunk in front of position 0
]


@pytest.mark.parametrize("qt,kvt", [(BF16, BF16), (F32, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("new,total,bt,nq,nkv,hd", SHAPES)
def test_chunk_attention_matches_fp64(A, new, total, bt, nq, nkv, hd, qt, kvt):
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    k, v, table, width, _ = pool(new, total, bt, nkv, hd, kvt, seed=sum(total) + nq)
    q = torch.randn(starts[-1] + 2, nq * hd, generator=torch.Generator().manual_seed(5)).to(qt)  # two rows of padding
    scale = 1.0 / math.sqrt(hd)
    got, ws = run_attn(A, q, k, v, table, starts, total, bt, nq, nkv, hd, scale, width)
    assert A.ds_workspace_error(ws) == 0
    assert (got[starts[-1]:] == 7).all()  # rows behind the last sequence stay
    want, d, vmax = attn_reference(q[:starts[-1]], k, v, table, starts, total, bt, nq, nkv, hd, scale)
    attn_near(got[:starts[-1]], want, d, vmax, max(total), nq, hd, qt == BF16)
    again, _ = run_attn(A, q, k, v, table, starts, total, bt, nq, nkv, hd, scale, width, ws=ws)
    assert torch.equal(got, again)  # the workspace is ready again, and the same bits come out


@pytest.mark.parametrize("qt,kvt", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("new,total,bt,nq,nkv,hd", [
    ([1] * 6, [5, 64, 65, 129, 700, 1], 16, 16, 4, 128),
    ([1, 2, 1], [300, 2, 64], 5, 4, 4, 64),
    ([2, 1, 3, 1], [90, 513, 200, 128], 16, 6, 2, 80),
    ([1, 1], [256, 77], 16, 8, 1, 256),
    ([0] * 15 + [1] + [0] * 15, [3] * 15 + [140] + [9] * 15, 16, 24, 1, 64),   # groups of 24, most sequences without rows
    ([1] * 30 + [61] + [1] * 30, [20] * 30 + [333] + [70] * 30, 16, 8, 4, 128),  # a chunk among single tokens
    ([3, 1, 1], [2, 0, 9], 16, 4, 2, 4),                                        # rows that attend nothing
])
def test_chunk_attention_with_few_rows_a_sequence(A, new, total, bt, nq, nkv, hd, qt, kvt):
    """16 (row, head) pairs a sequence or fewer on average: the plain cores' small tiles."""
    assert (sum(new) + 2) * (nq // nkv) <= 16 * len(new)
    test_chunk_attention_matches_fp64(A, new, total, bt, nq, nkv, hd, qt, kvt)


def test_chunk_attention_contiguous_slots(A):
    new, total, bt, nq, nkv, hd = [5, 80], [100, 90], 16, 8, 2, 128
    k, v, table, width, _ = pool(new, total, bt, nkv, hd, BF16, 3, paged=False)
    q = torch.randn(85, nq * hd).to(BF16)
    a, _ = run_attn(A, q, k, v, table, [0, 5, 85], total, bt, nq, nkv, hd, 0.1, width, paged=False)
    b, _ = run_attn(A, q, k, v, table, [0, 5, 85], total, bt, nq, nkv, hd, 0.1, width)
    assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("qt,kvt,bt", [(BF16, BF16, 16), (F32, BF16, 16), (F32, F32, 16), (BF16, BF16, 64)])
def test_what_a_row_does_not_attend_does_not_reach_it(A, qt, kvt, bt, bad):
    """Positions past the length, past a row's own, blocks of no sequence: NaN and infinities there change no bit."""
    new, total, nq, nkv, hd = [40, 1, 9], [171, 77, 9], 8, 2, 128
    starts = [0, 40, 41, 50]
    k, v, table, width, rows = pool(new, total, bt, nkv, hd, kvt, 11)
    q = torch.randn(50, nq * hd, generator=torch.Generator().manual_seed(6)).to(qt)
    clean, _ = run_attn(A, q, k, v, table, starts, total, bt, nq, nkv, hd, 0.1, width)
    seen = torch.zeros(rows, dtype=torch.bool)
    for s in range(3):
        seen[slots_of(table, s, total[s], bt)] = True
    k2, v2 = k.clone(), v.clone()
    k2[~seen], v2[~seen] = bad, bad
    got, _ = run_attn(A, q, k2, v2, table, starts, total, bt, nq, nkv, hd, 0.1, width)
    assert torch.equal(clean, got)
    # position 150 of sequence 0 is row 19's own: the rows before it do not attend it
    at = slots_of(table, 0, 151, bt)[150]
    k2, v2 = k.clone(), v.clone()
    k2[at], v2[at, 3] = bad, bad
    got, _ = run_attn(A, q, k2, v2, table, starts, total, bt, nq, nkv, hd, 0.1, width)
    assert torch.equal(clean[:19], got[:19]) and torch.equal(clean[40:], got[40:])
    # a non-finite value alone (k as it was) shows in its own column of the rows that attend it, and there only
    v2 = v.clone()
    v2[at, 3] = bad
    got, _ = run_attn(A, q, k, v2, table, starts, total, bt, nq, nkv, hd, 0.1, width)
    assert torch.equal(clean[:19], got[:19]) and torch.equal(clean[40:], got[40:])
    col = got[19:40].view(21, nq, hd)
    first = col[:, :nq // nkv, 3]
    assert (torch.isnan(first) if bad != bad else first == bad).all()
    col = col.clone()
    col[:, :nq // nkv, 3] = clean[19:40].view(21, nq, hd)[:, :nq // nkv, 3]
    assert torch.equal(col, clean[19:40].view(21, nq, hd))


def test_rows_with_all_scores_equal_or_far_apart(A):
    """Equal scores average the values; one score far above the others picks its value."""
    nq, nkv, hd, bt, T = 8, 2, 128, 16, 700
    k, v, table, width, _ = pool([3], [T], bt, nkv, hd, BF16, 4)
    q = torch.zeros(3, nq * hd, dtype=BF16)
    got, _ = run_attn(A, q, k, v, table, [0, 3], [T], bt, nq, nkv, hd, 0.1, width)
    want, d, vmax = attn_reference(q, k, v, table, [0, 3], [T], bt, nq, nkv, hd, 0.1)
    attn_near(got, want, d, vmax, T, nq, hd, True)
    at = slots_of(table, 0, T, bt)
    q = torch.full((3, nq * hd), 4.0, dtype=BF16)
    k[at] = -1.0
    k[at[333]] = 1.0   # 1024 * 0.1 above the others in log: their weights underflow to nothing
    got, _ = run_attn(A, q, k, v, table, [0, 3], [T], bt, nq, nkv, hd, 0.1, width)
    pick = v[at[333]].view(nkv, hd).repeat_interleave(nq // nkv, 0).reshape(-1)
    assert torch.equal(got.cpu(), pick.expand(3, -1))


def test_rising_scores_rescale_the_running_sum(A):
    """Scores that climb by whole units with the position: every step's maximum replaces the last one's."""
    nq, nkv, hd, bt, T = 4, 1, 128, 16, 1500
    k, v, table, width, _ = pool([2], [T], bt, nkv, hd, BF16, 8)
    at = slots_of(table, 0, T, bt)
    k[at] = 0.0
    k[at, 0] = (torch.arange(T) / 16.0).to(BF16)
    q = torch.zeros(2, nq * hd, dtype=BF16)
    q.view(2, nq, hd)[:, :, 0] = torch.tensor([1.0, 4.0, 0.25, -2.0]).to(BF16)
    got, _ = run_attn(A, q, k, v, table, [0, 2], [T], bt, nq, nkv, hd, 1.0, width)
    want, d, vmax = attn_reference(q, k, v, table, [0, 2], [T], bt, nq, nkv, hd, 1.0)
    attn_near(got, want, d, vmax, T, nq, hd, True)


def test_chunk_attention_is_the_decode_attention_for_single_tokens(A):
    new, total, bt, nq, nkv, hd = [1] * 6, [1, 40, 500, 1000, 16, 33], 16, 32, 8, 128
    k, v, table, width, _ = pool(new, total, bt, nkv, hd, BF16, 13)
    q = torch.randn(6, nq * hd)
    got, _ = run_attn(A, q, k, v, table, list(range(7)), total, bt, nq, nkv, hd, 0.088, width)
    out, ws = torch.empty(6, nq * hd, device="cuda"), A.workspace(A.ds_attention_workspace_bytes(6, nq, nkv, hd, width * bt))
    A.ds_gqa_decode_attn(q.cuda(), k.cuda(), v.cuda(), k.shape[0], table.cuda(), width, bt, i32(total), 6, nq, nkv, hd,
                         0.088, out, ws)
    assert (got - out).abs().max() <= 1e-4 * out.abs().max()  # the decode attention's own tolerance


def test_bad_device_values_are_clamped_and_flagged(A):
    nq, nkv, hd, bt = 8, 2, 128, 16
    k, v, table, width, rows = pool([4, 4], [60, 20], bt, nkv, hd, BF16, 2)
    q = torch.randn(8, nq * hd).to(BF16)
    for starts, total, change in [([0, 4, 99], [60, 20], None), ([0, 4, 8], [60, 99999], None),
                                  ([0, 4, 8], [-5, 20], None), ([0, 6, 4], [60, 20], None),
                                  ([0, 4, 8], [60, 20], (0, 1, rows)), ([0, 4, 8], [60, 20], (1, 0, -1))]:
        t = table.clone()
        if change:
            t[change[0], change[1]] = change[2]
        got, ws = run_attn(A, q, k, v, t, starts, total, bt, nq, nkv, hd, 0.1, width)
        assert A.ds_workspace_error(ws) == A.DS_ERR_POSITION
        assert torch.isfinite(got.float()).all()
        _, _ = run_attn(A, q, k, v, table, [0, 4, 8], [60, 20], bt, nq, nkv, hd, 0.1, width, ws=ws)
        assert A.ds_workspace_error(ws) == 0


def test_two_streams_with_a_workspace_each(A):
    new, total, bt, nq, nkv, hd = [3, 100], [700, 260], 16, 8, 2, 128
    k, v, table, width, _ = pool(new, total, bt, nkv, hd, BF16, 21)
    k, v, table = k.cuda(), v.cuda(), table.cuda()
    q = torch.randn(103, nq * hd).to(BF16).cuda()
    want, _ = run_attn(A, q, k, v, table, [0, 3, 103], total, bt, nq, nkv, hd, 0.1, width)
    starts, lens = i32([0, 3, 103]), i32(total)
    torch.cuda.synchronize()
    outs = []
    for _ in range(2):
        st = torch.cuda.Stream()
        out = torch.zeros_like(q)
        ws = A.workspace(A.ds_chunk_attention_workspace_bytes(2, 103, nq, nkv, hd))
        torch.cuda.synchronize()
        outs.append((st, out, ws))
    for _ in range(20):
        for st, out, ws in outs:
            A.ds_gqa_chunk_attn(q, 103, starts, lens, 2, k, v, k.shape[0], table, width, bt, nq, nkv, hd, 0.1, out, ws,
                                stream=st)
    torch.cuda.synchronize()
    for _, out, ws in outs:
        assert torch.equal(out, want) and A.ds_workspace_error(ws) == 0


# --------------------------------------------------------------- together
@pytest.mark.parametrize("cache,qt", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("graph", [False, True])
def test_a_serving_loop(A, cache, qt, graph):
    """Steps of chunks and single tokens through plan, rope and attention, eagerly or as one captured graph replayed
    with new lengths: every row equals attention over the sequence's own history, held apart in fp64."""
    nq, nkv, hd, bt, width, blocks, n, rows = 8, 2, 64, 16, 12, 40, 4, 96
    scale, base = 0.125, 10000.0
    steps = [[40, 3, 0, 17], [1, 30, 5, 1], [1, 1, 50, 1], [1, 1, 1, 1], [0, 2, 33, 1]]
    g = torch.Generator().manual_seed(3)
    cached, new = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    free, at = i32(np.random.RandomState(1).permutation(blocks)), 0
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    o = {k: torch.zeros(m, dtype=torch.int32, device="cuda") for k, m in
         (("starts", n + 1), ("lens", n), ("row_seq", rows), ("pos", rows), ("slots", rows), ("taken", 1))}
    x = torch.zeros(rows, (nq + 2 * nkv) * hd, device="cuda")
    k, v = (torch.zeros(blocks * bt, nkv * hd, dtype=cache, device="cuda") for _ in range(2))
    q, out = (torch.zeros(rows, nq * hd, dtype=qt, device="cuda") for _ in range(2))
    ws = [A.workspace(256), A.workspace(256), A.workspace(A.ds_chunk_attention_workspace_bytes(n, rows, nq, nkv, hd))]

    def step(stream=None):
        A.ds_paged_plan(cached, new, n, free, bt, blocks * bt, table, width, o["starts"], o["lens"], o["row_seq"],
                        o["pos"], o["slots"], rows, o["taken"], ws[0], stream=stream)
        A.ds_rope_append(x, x.shape[1], rows, o["pos"], 1, None, nq, nkv, hd, hd, base, 0, q, k, v, blocks * bt,
                         o["slots"], ws[1], stream=stream)
        A.ds_gqa_chunk_attn(q, rows, o["starts"], o["lens"], n, k, v, blocks * bt, table, width, bt, nq, nkv, hd, scale,
                            out, ws[2], stream=stream)

    if graph:
        step()  # with no new rows: every kernel is loaded before the capture
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
    hist = [[np.zeros((0, nkv, hd))] * 2 for _ in range(n)]
    for m in steps:
        total = sum(m)
        xh = torch.randn(total, x.shape[1], generator=g)
        x[:total] = xh.cuda()
        new.copy_(i32(m))
        out.fill_(7.0)
        cg.replay() if graph else step()
        torch.cuda.synchronize()
        assert [A.ds_workspace_error(w) for w in ws] == [0, 0, 0]
        assert (out[total:] == 7).all()
        taken = int(o["taken"])
        free[:blocks - at - taken] = free[taken:blocks - at].clone()  # what is left moves to the front
        at += taken
        pos = np.concatenate([int(cached[s]) + np.arange(m[s]) for s in range(n)])
        want, _ = rope_reference(xh, pos[None], np.zeros(hd // 2, int), nq, nkv, hd, hd, base, 0)
        r = 0
        for s in range(n):
            # the history as the cache holds it: rounded to its type
            kk, vv = (torch.from_numpy(want[r:r + m[s], a:a + nkv]).to(cache).double().numpy() for a in (nq, nq + nkv))
            hist[s] = [np.concatenate([h, w]) for h, w in zip(hist[s], (kk, vv))]
            for j in range(m[s]):
                seen = int(cached[s]) + j + 1
                qq = torch.from_numpy(want[r + j, :nq]).to(qt).double().numpy()
                kk, vv = (np.repeat(h[:seen], nq // nkv, 1) for h in hist[s])
                e = np.einsum("hd,thd->ht", qq, kk) * scale
                w = np.exp(e - e.max(1, keepdims=True))
                ref = np.einsum("ht,thd->hd", w / w.sum(1, keepdims=True), vv).reshape(-1)
                # q and k differ from the reference's by a flipped rounding of their type at most (a whole step, 2
                # halves each, of |q||k| scale in the score), v likewise; weights and output as in the bound above
                t = max(H if cache == BF16 else 16 * U, H if qt == BF16 else 16 * U)
                ds = 4 * t * scale * np.einsum("hd,thd->ht", abs(qq), abs(kk)).max()
                bound = (2 * ds + 4 * t) * abs(vv).max()
                got = out[r + j].double().cpu().numpy()
                assert np.abs(got - ref).max() <= bound
                # and in the mean, where flips are rare, the result is near
                assert np.sqrt(np.mean((got - ref) ** 2)) <= 4 * t * np.sqrt(np.mean(vv ** 2))
            r += m[s]
        cached += new


# ------------------------------------------------- larger and longer batches
def attn_reference_fast(q, k, v, table, starts, total, bt, nq, nkv, hd, scale):
    """attn_reference in matrices on the GPU (still 64 bits), for batches too large for its loops."""
    out = torch.zeros(q.shape[0], nq, hd, dtype=torch.float64, device="cuda")
    d, vmax = torch.zeros(q.shape[0], nq, 1, dtype=torch.float64), torch.zeros(q.shape[0], nq, 1, dtype=torch.float64)
    q, k, v, table = q.cuda(), k.cuda(), v.cuda(), table.cuda()
    for s in range(len(total)):
        n, L = starts[s + 1] - starts[s], total[s]
        if n == 0:
            continue
        t = torch.arange(L, device="cuda")
        at = table[s].long()[t // bt] * bt + t % bt
        ks, vs = (x[at].double().view(L, nkv, hd).repeat_interleave(nq // nkv, 1) for x in (k, v))
        qs = q[starts[s]:starts[s + 1]].double().view(n, nq, hd)
        e = torch.einsum("jhd,thd->hjt", qs, ks) * scale
        hidden = t[None, :] > (L - n + torch.arange(n, device="cuda"))[:, None]
        w = torch.softmax(e.masked_fill(hidden, -math.inf), 2)
        out[starts[s]:starts[s + 1]] = torch.einsum("hjt,thd->jhd", w, vs)
        # bounds over all of the sequence's positions: no smaller than the row's own
        mag = (qs.abs().sum(2) * ks.abs().amax()).cpu()
        d[starts[s]:starts[s + 1], :, 0] = (hd + 4) * U * scale * mag
        vmax[starts[s]:starts[s + 1]] = float(vs.abs().max())
    return out.view(q.shape[0], -1).cpu(), d, vmax


@pytest.mark.parametrize("qt", [BF16, F32])
@pytest.mark.parametrize("kind", ["many short", "one long", "chunks", "narrow heads", "prompt"])
def test_chunk_attention_on_larger_batches(A, kind, qt):
    g = np.random.RandomState(7)
    if kind == "many short":  # more sequences than a block has threads, some without rows
        new = g.randint(0, 5, 900)
        total, bt, nq, nkv, hd = new + g.randint(0, 200, 900), 8, 4, 2, 64
        total = np.maximum(total, 1)
    elif kind == "one long":  # a tile shared by most of the CTAs
        new, total, bt, nq, nkv, hd = np.array([3]), np.array([30011]), 32, 8, 2, 128
    elif kind == "chunks":
        new = np.array([1, 257, 1, 64, 65, 1, 129, 0, 300, 1])
        total, bt, nq, nkv, hd = new + np.array([2000, 700, 1, 0, 63, 128, 512, 9, 1111, 4095]), 16, 32, 8, 128
    elif kind == "narrow heads":
        new = g.randint(1, 90, 40)
        total, bt, nq, nkv, hd = new + g.randint(0, 900, 40), 64, 14, 2, 64
    else:
        new, total, bt, nq, nkv, hd = np.array([1537]), np.array([1600]), 16, 8, 1, 128
    new, total = new.tolist(), total.tolist()
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    k, v, table, width, _ = pool(new, total, bt, nkv, hd, BF16, seed=3)
    q = torch.randn(starts[-1], nq * hd, generator=torch.Generator().manual_seed(9)).to(qt)
    scale = 1.0 / math.sqrt(hd)
    got, ws = run_attn(A, q, k, v, table, starts, total, bt, nq, nkv, hd, scale, width)
    assert A.ds_workspace_error(ws) == 0
    want, d, vmax = attn_reference_fast(q, k, v, table, starts, total, bt, nq, nkv, hd, scale)
    attn_near(got, want, d, vmax, max(total), nq, hd, qt == BF16)
    for _ in range(3):  # the same bits from every run
        again, _ = run_attn(A, q, k, v, table, starts, total, bt, nq, nkv, hd, scale, width, ws=ws)
        assert torch.equal(got, again)


@pytest.mark.parametrize("qt", [BF16, F32])
def test_many_tiles_with_values_that_are_not_finite(A, qt):
    """A non-finite value in the new rows of every sequence: tiles of both kinds, one after the other in every CTA, keep
    theirs apart, and a clean batch through the same workspace afterwards is what it was before."""
    g = np.random.RandomState(5)
    n, bt, nq, nkv, hd = 60, 16, 8, 2, 128
    new = g.randint(1, 120, n)
    total = (new + g.randint(0, 300, n)).tolist()
    new = new.tolist()
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    k, v, table, width, _ = pool(new, total, bt, nkv, hd, BF16, seed=13)
    q = torch.randn(starts[-1], nq * hd, generator=torch.Generator().manual_seed(2)).to(qt)
    clean, ws = run_attn(A, q, k, v, table, starts, total, bt, nq, nkv, hd, 0.1, width)
    v2 = v.clone()
    at_row = [int(g.randint(0, m)) for m in new]
    col = [int(g.randint(0, nkv * hd)) for _ in new]
    bad = [(float("nan"), float("inf"), float("-inf"))[s % 3] for s in range(n)]
    for s in range(n):
        t = total[s] - new[s] + at_row[s]
        v2[int(table[s, t // bt]) * bt + t % bt, col[s]] = bad[s]
    got, _ = run_attn(A, q, k, v2, table, starts, total, bt, nq, nkv, hd, 0.1, width, ws=ws)
    want = clean.clone().view(-1, nkv, nq // nkv, hd)
    for s in range(n):
        want[starts[s] + at_row[s]:starts[s + 1], col[s] // hd, :, col[s] % hd] = bad[s]
    want = want.view_as(clean)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])
    again, _ = run_attn(A, q, k, v, table, starts, total, bt, nq, nkv, hd, 0.1, width, ws=ws)
    assert torch.equal(clean, again) and A.ds_workspace_error(ws) == 0


def test_offsets_past_32_bits(A):
    """A pool of more than 2^31 elements: rows at its end are written and read where they belong."""
    nq, nkv, hd, bt = 16, 8, 128, 16
    rows = (1 << 21) + 1024            # x 1,024 elements
    k = torch.zeros(rows, nkv * hd, dtype=BF16, device="cuda")
    v = torch.zeros(rows, nkv * hd, dtype=BF16, device="cuda")
    T, width = 200, 13
    blocks = rows // bt
    table = torch.tensor([[blocks - 1 - i for i in range(width)]], dtype=torch.int32)
    x = torch.randn(T, (nq + 2 * nkv) * hd, generator=torch.Generator().manual_seed(4))
    t = torch.arange(T)
    slots = (table[0].long()[t // bt] * bt + t % bt).to(torch.int32)
    for qt in (BF16, F32):
        q = torch.zeros(T, nq * hd, dtype=qt, device="cuda")
        A.ds_rope_append(x.cuda(), x.shape[1], T, t.to(torch.int32).cuda(), 1, None, nq, nkv, hd, hd, 1e4, 0, q, k, v,
                         rows, slots.cuda(), A.workspace(256))
        at = slots.long().cuda()
        assert torch.equal(v[at], x[:, (nq + nkv) * hd:].to(BF16).cuda())
        assert not v[:rows - width * bt].any() and not k[:rows - width * bt].any()
        out = torch.zeros_like(q)
        ws = A.workspace(A.ds_chunk_attention_workspace_bytes(1, T, nq, nkv, hd))
        A.ds_gqa_chunk_attn(q, T, i32([0, T]), i32([T]), 1, k, v, rows, table.cuda(), width, bt, nq, nkv, hd, 0.1, out, ws)
        want, d, vmax = attn_reference_fast(q, k, v, table, [0, T], [T], bt, nq, nkv, hd, 0.1)
        attn_near(out, want, d, vmax, T, nq, hd, qt == BF16)
        assert A.ds_workspace_error(ws) == 0


def test_two_captured_graphs_replayed_at_once(A):
    """Two captured calls with a workspace each, replayed on two streams without waiting for one another."""
    new, total, bt, nq, nkv, hd = [1, 90, 1, 1], [1500, 333, 4000, 17], 16, 32, 8, 128
    starts = [0, 1, 91, 92, 93]
    k, v, table, width, _ = pool(new, total, bt, nkv, hd, BF16, 31)
    k, v, table = k.cuda(), v.cuda(), table.cuda()
    st, ln = i32(starts), i32(total)
    calls = []
    for qt in (BF16, F32):
        q = torch.randn(93, nq * hd, device="cuda").to(qt)
        want, _ = run_attn(A, q, k, v, table, starts, total, bt, nq, nkv, hd, 0.09, width)
        out, ws = torch.zeros_like(q), A.workspace(A.ds_chunk_attention_workspace_bytes(4, 93, nq, nkv, hd))
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            for _ in range(5):
                A.ds_gqa_chunk_attn(q, 93, st, ln, 4, k, v, k.shape[0], table, width, bt, nq, nkv, hd, 0.09, out, ws)
        calls.append((cg, q, out, ws, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(6):
        for cg, _, _, _, _, s in calls:
            with torch.cuda.stream(s):
                cg.replay()
    torch.cuda.synchronize()
    for _, _, out, ws, want, _ in calls:
        assert torch.equal(out, want) and A.ds_workspace_error(ws) == 0
