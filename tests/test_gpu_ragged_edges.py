"""Edges of the ragged-step operators on the GPU."""
import math
import threading
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and bf16, relative to the value
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from autoregressive_decode_step_gb300 import abi
    return abi


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


@pytest.mark.parametrize("qt,kvt", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 60])
def test_an_infinite_key_that_a_row_attends(A, new, hd, qt, kvt):
    """q . k is an infinity of q's sign times k's: minus infinity takes the
    position out of the row's sum, plus infinity makes the row NaN, whatever
    digits q has.

    Tolerance: two scores' error d each and (T + 8) u over the sum, H for bf16
    weights, and the output's rounding, as for finite keys."""
    T, nq, nkv = new + 37, 4, 2
    g = torch.Generator().manual_seed(new + hd)
    q = torch.randn(new, nq, hd, generator=g).to(qt)
    q[:, 0] = 1.0              # numbers of few digits, and of one sign
    q[:, 1] = q[:, 1].abs()
    q[:, 2] = -0.40625
    q[:, 3] = -q[:, 3].abs()
    k, v = (torch.randn(112, nkv, hd, generator=g).to(kvt) for _ in range(2))
    k[5, :, 3], k[11, 0, hd - 1], k[20, 1, 7] = -math.inf, -math.inf, math.inf
    scale = 1.0 / math.sqrt(hd)
    out, ws = torch.full((new, nq * hd), 7.0, dtype=qt, device="cuda"), A.workspace(
        A.ds_chunk_attention_workspace_bytes(1, new, nq, nkv, hd))
    A.ds_gqa_chunk_attn(q.view(new, -1).cuda(), new, i32([0, new]), i32([T]), 1, k.view(112, -1).cuda(),
                        v.view(112, -1).cuda(), 112, None, 7, 16, nq, nkv, hd, scale, out, ws)
    kk, vv = (x[:T].double().repeat_interleave(nq // nkv, 1) for x in (k, v))
    e = (q.double()[:, None] * kk[None]).sum(3).permute(2, 0, 1) * scale
    e = e.masked_fill(torch.arange(T) > T - new + torch.arange(new)[:, None], -math.inf)
    w = torch.softmax(e, 2)
    want = torch.einsum("hjt,thd->jhd", w, vv)
    finite = torch.where(torch.isfinite(kk), kk, 0.0).abs()
    d = (hd + 4) * U * scale * torch.einsum("jhd,thd->jht", q.double().abs(), finite).amax(2)[:, :, None]
    half = U if qt == F32 else H
    slack = (2 * d + (T + 8) * U + (H if qt == BF16 else 0)) * vv.abs().max()
    got = out.double().cpu().view(new, nq, hd)
    assert not torch.isnan(want[:, :2]).any() and torch.isnan(want[:, 2:]).all()  # heads 2 and 3: plus infinity
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    err = (got - want).abs()[:, :2]
    assert (err <= (slack + half * (want.abs() + slack))[:, :2]).all(), float(err.max())
    assert A.ds_workspace_error(ws) == 0


@pytest.mark.parametrize("qt,kvt", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("T", [1, 130, 700])
def test_a_row_with_every_score_minus_infinity_is_nan(A, T, qt, kvt):
    """No weight is left to divide by, whatever the values are: infinite ones do not show as infinities."""
    nq, nkv, hd = 4, 2, 64
    q = torch.ones(1, nq * hd, dtype=qt, device="cuda")
    k, v = (torch.randn(704, nkv * hd, device="cuda").to(kvt) for _ in range(2))
    k[:, 5] = -math.inf                     # every key of the first head
    v[0, 3], v[T - 1, 9], v[0, hd + 3] = math.inf, -math.inf, math.inf
    out = torch.zeros_like(q)
    ws = A.workspace(A.ds_chunk_attention_workspace_bytes(1, 1, nq, nkv, hd))
    A.ds_gqa_chunk_attn(q, 1, i32([0, 1]), i32([T]), 1, k, v, 704, None, 44, 16, nq, nkv, hd, 0.125, out, ws)
    got = out.view(nq, hd)
    assert torch.isnan(got[:2]).all()
    assert (got[2:, 3] == math.inf).all() and torch.isfinite(got[2:, 4:]).all()


@pytest.mark.parametrize("base", [1e-3, 10000.0, 500000.0, 1e6])
@pytest.mark.parametrize("hd,rot,layout", [(128, 128, 0), (256, 256, 1), (96, 80, 1), (6, 6, 0)])
def test_angles_of_far_positions(A, hd, rot, layout, base):
    """Pairs (1, 0) come out as cosine and sine of the angle, here worked out in 60 digits. Tolerance: 2^-33 of a turn,
    and 4 u for the fp32 argument (an eighth of a turn at most) and the two functions; 1 c - 0 s is exact."""
    getcontext().prec = 60
    pi = Decimal("3.141592653589793238462643383279502884197169399375105820974944592307816406286209")
    pos = [2 ** 31 - 1, 2 ** 31 - 77, 2 ** 30 + 12345, 99999989, 6000000, 131071, 0]
    n = len(pos)
    x = torch.zeros(n, 3, hd, device="cuda")
    first = slice(0, rot // 2) if layout == 0 else slice(0, rot, 2)
    second = slice(rot // 2, rot) if layout == 0 else slice(1, rot, 2)
    x[:, :, first] = 1.0
    q, k, v = (torch.zeros(n, hd, device="cuda") for _ in range(3))
    ws = A.workspace(A.ds_rope_append_workspace_bytes())
    A.ds_rope_append(x.view(n, -1), 3 * hd, n, i32([pos]), 1, None, 1, 1, hd, rot, base, layout, q, k, v, n,
                     i32(range(n)), ws)
    angle = np.array([[float(i * (Decimal(base) ** (Decimal(-2 * p) / rot)) % (2 * pi)) for p in range(rot // 2)]
                      for i in pos])
    for got in (q.double().cpu().numpy(), k.double().cpu().numpy()):
        assert np.abs(got[:, first] - np.cos(angle)).max() <= 4 * U + 2 * math.pi * 2.0 ** -33
        assert np.abs(got[:, second] - np.sin(angle)).max() <= 4 * U + 2 * math.pi * 2.0 ** -33


def test_rope_append_of_two_widths_from_two_threads(A):
    """Rows of two widths through one kernel (fp32 rows by bulk copies) from
    two host threads at once: every call is accepted and does its own work."""
    n, calls, errors = 2048, 500, []

    def make(nq, nkv):
        x = torch.randn(n, (nq + 2 * nkv) * 128, device="cuda")
        q = torch.zeros(n, nq * 128, device="cuda")
        k = torch.zeros(n, nkv * 128, device="cuda")
        pos, ws, st = torch.arange(n, dtype=torch.int32, device="cuda")[None], A.workspace(256), torch.cuda.Stream()
        return dict(x=x, q=q, k=k, v=torch.zeros_like(k), pos=pos, ws=ws, st=st, nq=nq, nkv=nkv)

    def call(o, q, k, v, ws, st=None):
        A.ds_rope_append(o["x"], o["x"].shape[1], n, o["pos"], 1, None, o["nq"], o["nkv"], 128, 128, 1e4, 0, q, k, v, n,
                         o["pos"][0], ws, stream=st)

    def work(o):
        try:
            for _ in range(calls):
                call(o, o["q"], o["k"], o["v"], o["ws"], o["st"])
        except Exception as e:
            errors.append(e)

    sets = [make(32, 8), make(4, 2)]
    want = []
    for o in sets:
        alone = [torch.zeros_like(o[t]) for t in "qkv"]
        call(o, *alone, A.workspace(256))
        want.append(alone)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(o,)) for o in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    for o, w in zip(sets, want):
        assert all(torch.equal(o[t], w[i]) for i, t in enumerate("qkv")) and A.ds_workspace_error(o["ws"]) == 0


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("qt", [BF16, F32])
def test_values_that_are_not_finite_in_tile_after_tile(A, hd, qt):
    """Several non-finite values in the new rows of each of 500 sequences, so that every CTA has a run of tiles of both
    kinds with values to set aside, split tiles among them: each comes out in its own column of the rows that attend it,
    every other element as from the clean batch, time after time."""
    g = np.random.RandomState(hd)
    n, bt, nq, nkv = 500, 16, 8, 2
    new = g.randint(1, 150, n)
    total = new + g.randint(0, 200, n)
    starts = np.concatenate([[0], np.cumsum(new)])
    width = int(-(-total.max() // bt))
    table = torch.from_numpy(g.permutation(n * width).astype(np.int32)).view(n, width)
    gen = torch.Generator().manual_seed(hd + 1)
    k, v = (torch.randn(n * width * bt, nkv * hd, generator=gen).to(BF16) for _ in range(2))
    q = torch.randn(int(starts[-1]), nq * hd, generator=gen).to(qt).cuda()
    bad_v, marks = v.clone(), []
    for s in range(n):
        for i in range(g.randint(0, 5)):
            t = int(g.randint(total[s] - new[s], total[s]))
            col, x = int(g.randint(0, nkv * hd)), (math.nan, math.inf, -math.inf)[g.randint(3)]
            if all((s, col) != m[:2] for m in marks):
                bad_v[int(table[s, t // bt]) * bt + t % bt, col] = x
                marks.append((s, col, int(starts[s] + t - (total[s] - new[s])), x))
    ws = A.workspace(A.ds_chunk_attention_workspace_bytes(n, q.shape[0], nq, nkv, hd))
    args = i32(starts), i32(total), n, k.cuda()
    vs, vb, tb = v.cuda(), bad_v.cuda(), table.cuda()

    def call(values):
        out = torch.full_like(q, 7.0)
        A.ds_gqa_chunk_attn(q, q.shape[0], *args, values, k.shape[0], tb, width, bt, nq, nkv, hd, 0.1, out, ws)
        return out

    clean = call(vs)
    want = clean.clone().view(-1, nkv, nq // nkv, hd)
    for s, col, row, x in marks:
        want[row:int(starts[s + 1]), col // hd, :, col % hd] = x
    want = want.view_as(clean)
    for _ in range(5):
        got = call(vb)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got, 0.0), torch.nan_to_num(want, 0.0))
    assert torch.equal(call(vs), clean) and A.ds_workspace_error(ws) == 0


# ------------------------------------------------------- the digits of fp32 q
PIECE_CASES = [(0.25, 4), (2.0, 2), (4.0, 8)]  # largest score, positions


def piece_data(smax, T, n_seqs, nq, nkv, hd):
    """q with one element a head that is not zero, so that a score is one product and its error a few roundings;
    values 1 and -1, so that an output's error is that of the weights."""
    g = torch.Generator().manual_seed(T + hd)
    q = torch.zeros(n_seqs, nq, hd)
    q[:, :, 5] = torch.rand(n_seqs, nq, generator=g) * 0.5 + 0.5
    k = torch.randn(n_seqs * T, nkv, hd, generator=g)
    k[:, :, 5] = (torch.rand(n_seqs * T, nkv, generator=g) * 2 - 1) * smax
    v = torch.where(torch.rand(n_seqs * T, nkv, hd, generator=g) < 0.5, -1.0, 1.0)
    return q, k.to(BF16), v.to(BF16)


def piece_bound(smax, T):
    """A score of three exact products: two sums, 2 u each if they are cut off, 4 u smax; times scale log2 e and from
    the maximum, 3 u of a difference of at most 2 smax; ex2.approx 4 u and a piece's cut u. Weights off by e move the
    mean of values +-1 by e at most. Then sums over T terms: products cut off (2 u), weights (u), three rows added, the
    reciprocal and its product, 8 u."""
    return (10 * smax + 5 + 3 * T + 8) * U


def pieces(x, n):
    """The first n of the bf16 numbers that add up to fp32 x, added."""
    total = torch.zeros_like(x, dtype=torch.float64)
    for _ in range(n):
        top = (x.view(torch.int32) & -65536).view(F32)
        total += top.double()
        x = x - top
    return total


def piece_reference(q, k, v, T, q_pieces=None, p_pieces=None):
    """fp64 attention of one row a sequence over its T positions (scale 1); with piece counts, what is left if the
    others were lost."""
    n, nq, hd = q.shape
    kk, vv = (x.double().view(n, T, -1, hd).repeat_interleave(nq // x.shape[1], 2) for x in (k, v))
    e = torch.einsum("nhd,nthd->nht", q.double() if q_pieces is None else pieces(q, q_pieces), kk)
    p = torch.exp(e - e.amax(2, keepdim=True))
    w = p if p_pieces is None else pieces(p.float(), p_pieces)
    return torch.einsum("nht,nthd->nhd", w, vv) / p.sum(2)[..., None]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("smax,T", PIECE_CASES)
def test_fp32_attention_keeps_fp32_digits(A, smax, T, hd):
    n, nq, nkv = 40, 8, 2
    q, k, v = piece_data(smax, T, n, nq, nkv, hd)
    bt = 8                                   # a block a sequence
    kc, vc = (torch.full((n, bt, nkv * hd), float("nan")).to(BF16) for _ in range(2))
    kc[:, :T], vc[:, :T] = k.view(n, T, -1), v.view(n, T, -1)
    out = torch.zeros(n, nq * hd, device="cuda")
    ws = A.workspace(A.ds_chunk_attention_workspace_bytes(n, n, nq, nkv, hd))
    A.ds_gqa_chunk_attn(q.view(n, -1).cuda(), n, i32(range(n + 1)), i32([T] * n), n, kc.view(n * bt, -1).cuda(),
                        vc.view(n * bt, -1).cuda(), n * bt, None, 1, bt, nq, nkv, hd, 1.0, out, ws)
    err = (out.double().cpu().view(n, nq, hd) - piece_reference(q, k, v, T)).abs().max()
    assert err <= piece_bound(smax, T), float(err) / U
