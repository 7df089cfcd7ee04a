"""ds_moe_layer against its formula in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3, F32, BF16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16
U = 2.0 ** -23  # one rounding or cut of an fp32 sum


@pytest.fixture(scope="module")
def abi():
    from autoregressive_decode_step_gb300 import build
    build.build()
    from autoregressive_decode_step_gb300 import abi as A
    return A


class Layer:
    def __init__(self, n, d, ff, experts, k, x=F32, w=BF16, router=BF16, norm=True, residual=False, seed=0, lean=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*s):
            return torch.randn(*s, generator=g, device="cuda")

        self.n, self.d, self.ff, self.e, self.k, self.norm = n, d, ff, experts, k, norm
        self.x = normal(n, d) * torch.exp(0.5 * normal(d))
        way = normal(d)
        self.x = (self.x + lean * way).to(x)
        self.router = (normal(experts, d) / math.sqrt(d) + lean * normal(experts)[:, None] * way / d).to(router)
        self.gs = self.ds = None
        self.gu, self.dn = normal(experts, 2, ff, d) / math.sqrt(d), normal(experts, d, ff) / math.sqrt(ff)
        if w == BF16:
            self.gu, self.dn = self.gu.to(w), self.dn.to(w)
        else:
            kb, fb = -(-d // 128), -(-ff // 128)
            self.gu, self.dn = (self.gu * 100).clamp(-448, 448).to(w), (self.dn * 100).clamp(-448, 448).to(w)
            self.gs = torch.exp(0.3 * normal(experts, 2, fb, kb)) / 100
            self.ds = torch.exp(0.3 * normal(experts, kb, fb)) / 100
        self.residual = normal(n, d).to(x) if residual else None

    def widened(self):
        gu, dn = self.gu.double(), self.dn.double()
        if self.gs is not None:
            gu = gu * self.gs.double().repeat_interleave(128, 2)[:, :, :self.ff].repeat_interleave(128, 3)[..., :self.d]
            dn = dn * self.ds.double().repeat_interleave(128, 1)[:, :self.d].repeat_interleave(128, 2)[..., :self.ff]
        return gu, dn

    def want(self):
        """(y, how far fp32 may be from it, ids, p) in 64 bits."""
        x = self.x.double()
        logits = x @ self.router.double().t()
        ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :self.k]
        p = torch.softmax(logits, 1).gather(1, ids)
        if self.norm:
            p = p / p.sum(1, keepdim=True)
        gu, dn = self.widened()
        y = torch.zeros_like(x) if self.residual is None else self.residual.double()
        far = 2.0 ** -24 * y.abs()
        # pieces: 24 bits of fp32 values, 16 of an intermediate before a bf16 output; before e4m3 weights no more than
        # a share of the largest of 128 (six pieces of a sixteenth each from 2^-10 on, beside 2^7: 2^-37, and so on)
        half = self.x.dtype == BF16
        piece, mid = 2.0 ** -24, 2.0 ** -16 if half else 2.0 ** -24
        tiny, tiny_mid = (0.0, 0.0) if self.gs is None else (2.0 ** -25, 2.0 ** -29) if half else (2.0 ** -37, 2.0 ** -37)

        def largest(v):
            b = torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % 128)).view(len(v), -1, 128).amax(2)
            return b.repeat_interleave(128, 1)[:, :v.shape[1]]
        for s in range(self.k):
            for e in ids[:, s].unique():
                at = (ids[:, s] == e).nonzero()[:, 0]
                a, g, u, w = x[at], gu[e, 0], gu[e, 1], dn[e]
                gate, up = a @ g.t(), a @ u.t()
                off = ((self.d + 16) * U + piece) * a.abs() + tiny * largest(a)
                dg, du = off @ g.abs().t(), off @ u.abs().t()
                act = gate * torch.sigmoid(gate)
                h = act * up
                # silu's slope is at most 1.1; exp, division and products round six times.  A product below
                # 2^-126 (a token of 1e-30 has gate and up of some 1e-26 each, so 1e-52) may become 0 in fp32.
                dh = 1.1 * dg * (up.abs() + du) + act.abs() * du + (6 * U + mid) * h.abs() + 2.0 ** -126
                dh = dh + tiny_mid * largest(h.abs() + dh)
                o = h @ w.t()
                do = dh @ w.abs().t() + (self.ff + 16) * U * ((h.abs() + dh) @ w.abs().t())
                q = p[at, s][:, None]
                y[at] = y[at] + q * o
                # p: exp of a difference, a sum over the experts, a division
                far[at] = far[at] + q * (do + (self.e + 8 + self.k) * U * (o.abs() + do)) + U * y[at].abs()
        return y, far, ids, p

    def run(self, abi, y=None, ws=None):
        y = torch.full_like(self.x, math.nan) if y is None else y
        ids = torch.full((self.n, self.k), -7, dtype=torch.int32, device="cuda")
        p = torch.full((self.n, self.k), math.nan, device="cuda")
        if ws is None:
            ws = abi.workspace(abi.ds_moe_layer_workspace_bytes(self.n, self.d, self.ff, self.e, self.k))
        abi.ds_moe_layer(self.x, self.router, self.k, self.norm, self.gu, self.gs, self.dn, self.ds, self.residual, y,
                         ids, p, ws)
        assert abi.ds_workspace_error(ws) == 0
        return y, ids, p

    def check(self, abi, **kw):
        y, ids, p = self.run(abi, **kw)
        want, far, wids, wp = self.want()
        assert torch.equal(ids.long(), wids)
        assert ((p - wp).abs() <= (self.e + 8 + self.k) * U * wp).all()
        if y.dtype == BF16:
            far = far + 2.0 ** -8 * (want.abs() + far)
        assert ((y.double() - want).abs() <= far).all()


SHAPES = [  # n, d, ff, experts, k
    (1, 16, 16, 1, 1), (1, 2048, 768, 128, 8), (2, 48, 80, 3, 2), (3, 128, 64, 60, 4), (5, 1008, 352, 7, 7),
    (8, 256, 128, 16, 1), (9, 512, 1024, 8, 2), (16, 144, 2000, 300, 16), (17, 640, 320, 4, 2), (33, 272, 208, 2, 2),
    (64, 1024, 256, 128, 8), (100, 128, 128, 1, 1), (256, 400, 144, 5, 3), (256, 64, 64, 512, 8)]


@pytest.mark.parametrize("x", [F32, BF16])
@pytest.mark.parametrize("w", [BF16, E4M3])
@pytest.mark.parametrize("shape", SHAPES)
def test_layer(abi, shape, w, x):
    i = SHAPES.index(shape)
    Layer(*shape, x=x, w=w, router=F32 if i % 3 == 0 else BF16, norm=i % 2 == 0, residual=i % 4 < 2, seed=i).check(abi)


@pytest.mark.parametrize("w", [BF16, E4M3])
def test_layer_favourites(abi, w):
    """Most tokens choose the same experts: more than one group of 32 tokens for one, none for another."""
    Layer(200, 256, 192, 16, 2, w=w, lean=3.0, seed=3).check(abi)


@pytest.mark.parametrize("d,ff", [(8, 8), (24, 1000), (1000, 24), (136, 72)])
def test_layer_multiples_of_eight(abi, d, ff):
    Layer(6, d, ff, 9, 3, seed=d, residual=True).check(abi)


@pytest.mark.parametrize("w", [BF16, E4M3])
def test_layer_digits(abi, w):
    """Short sums, where a lost piece of an fp32 value (2^-8 or 2^-11 of it) is far beyond the bound."""
    for seed in range(4):
        Layer(40, 16, 16, 4, 2, w=w, seed=seed).check(abi)


@pytest.mark.parametrize("x", [F32, BF16])
def test_layer_sizes_within_a_block(abi, x):
    """e4m3 experts, activations of very different sizes within 128 values, a zero token, a large one."""
    a = Layer(6, 256, 128, 4, 2, x=x, w=E4M3, seed=9)
    a.x *= torch.exp(4 * torch.randn(256, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")).to(x)
    a.x[2] = 0
    a.x[3] *= 1e-30
    a.x[4] *= 1e4
    a.router *= 1e-3
    a.check(abi)


def test_layer_ties_and_far_apart(abi):
    """Equal logits go to the lower index; logits that differ in the last bits of 64 are told apart."""
    a = Layer(4, 64, 32, 40, 5, router=F32, seed=2)
    a.router[:] = a.router[0]
    a.x[1] = 0
    y, ids, p = a.run(abi)
    assert torch.equal(ids.cpu(), torch.arange(5, dtype=torch.int32).repeat(4, 1))
    assert torch.equal(p, torch.full_like(p, 0.2))
    a.x[:] = 1
    a.router[:] = 2.0 ** 12
    a.router[33, 0] += 2.0 ** -11  # 2^-11 beside a sum of 2^18: lost in a plain fp32 sum
    a.router[7, 63] += 2.0 ** -10
    a.norm = True
    _, ids, _ = a.run(abi)
    assert torch.equal(ids.cpu(), torch.tensor([7, 33, 0, 1, 2], dtype=torch.int32).repeat(4, 1))


@pytest.mark.parametrize("w", [BF16, E4M3])
def test_layer_not_finite(abi, w):
    """A token with a NaN or an infinity: its own outputs alone, ids in range."""
    a = Layer(7, 256, 128, 6, 2, w=w, seed=4)
    good, _, _ = a.run(abi)
    a.x[2, 5], a.x[4, 200] = math.nan, math.inf
    y, ids, p = a.run(abi)
    assert ((ids >= 0) & (ids < 6)).all()
    assert not torch.isfinite(y[[2, 4]]).any() and not torch.isfinite(p[[2, 4]]).any()
    rest = [0, 1, 3, 5, 6]
    # which tokens share an expert changes no token's sums
    assert torch.equal(y[rest], good[rest])


def test_layer_in_place_and_without_extras(abi):
    a = Layer(12, 320, 160, 8, 2, residual=True, seed=6)
    want, ids, p = a.run(abi)
    space = abi.workspace(abi.ds_moe_layer_workspace_bytes(a.n, a.d, a.ff, a.e, a.k))
    for y in (a.residual.clone(), a.x.clone()):
        x, res = (a.x, y) if torch.equal(y, a.residual) else (y, a.residual)
        abi.ds_moe_layer(x, a.router, a.k, a.norm, a.gu, None, a.dn, None, res, y, None, None, space)
        assert torch.equal(y, want)


def test_layer_same_each_time_and_a_workspace_for_many(abi):
    shapes = [(1, 2048, 768, 128, 8), (64, 512, 256, 8, 2), (7, 1000, 344, 60, 4), (33, 128, 640, 3, 3)]
    space = abi.workspace(max(abi.ds_moe_layer_workspace_bytes(*s) for s in shapes))
    layers = [Layer(*s, seed=i) for i, s in enumerate(shapes)]
    first = [a.run(abi, ws=space)[0] for a in layers]
    for _ in range(3):
        for a, y in zip(layers, first):
            assert torch.equal(a.run(abi, ws=space)[0], y)


def test_layer_captured_and_on_two_streams(abi):
    a = Layer(16, 512, 256, 32, 4, seed=8)
    b = Layer(16, 512, 256, 32, 4, seed=8)
    spaces = [abi.workspace(abi.ds_moe_layer_workspace_bytes(a.n, a.d, a.ff, a.e, a.k)) for _ in range(2)]
    y = torch.empty_like(a.x)
    args = (a.router, a.k, a.norm, a.gu, None, a.dn, None, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        abi.ds_moe_layer(a.x, *args, y, None, None, spaces[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            abi.ds_moe_layer(a.x, *args, y, None, None, spaces[0])
    torch.cuda.synchronize()
    for seed in range(3):
        b.x = torch.randn(a.n, a.d, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
        a.x.copy_(b.x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.run(abi)[0], y)
    outs = [[torch.empty_like(y) for _ in range(10)] for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                abi.ds_moe_layer(a.x, *args, outs[k][i], None, None, spaces[k])
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for out in outs for o in out)
    assert all(abi.ds_workspace_error(s) == 0 for s in spaces)


def test_layer_offsets_past_32_bits(abi):
    """Experts' matrices of more than 2^32 bytes, the last expert chosen."""
    e, d, ff = 300, 2048, 2048
    one, many = Layer(2, d, ff, 1, 1, seed=5), Layer(2, d, ff, 1, 1, seed=5)
    many.e = e
    many.gu = torch.zeros(e, 2, ff, d, dtype=BF16, device="cuda")
    many.dn = torch.zeros(e, d, ff, dtype=BF16, device="cuda")
    many.gu[-1], many.dn[-1] = one.gu[0], one.dn[0]
    many.router = torch.zeros(e, d, dtype=BF16, device="cuda")
    many.router[-1] = one.x.sign().sum(0).to(BF16)
    y, ids, _ = many.run(abi)
    assert (ids == e - 1).all()
    want, far, _, _ = one.want()
    assert ((y.double() - want).abs() <= far).all()
