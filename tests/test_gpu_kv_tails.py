"""Attention over the paged 8-bit cache where one token holds much of the softmax, or one
page has a much larger value scale, before a long flat tail: the tail's weights are small
beside the row's largest one, and together they are much of the output.

The bound on the output has no term that grows with the number of visible tokens but that
of fp32 sums (o: output, w_j: weights, sum 1, v_j: values, size = sum_j w_j |v_j|):
  - one rounding to bf16, 2^-8 |o|;
  - a weight held as two e4m3 numbers, 2^-4 * 2^-4 of itself, by way of f16, 2^-12 (in f16
    alone: 2^-11): (2^-8 + 2^-12) size;
  - below their normal ranges, per weight: the two numbers 2^-22 of the largest weight of the same 32
    tokens, in powers of two with the value scale taken in (a block of 32 is held within
    (2^7, 2^8], the second number's smallest step is 2^-9 * 2^-5, half of it counts);
    (the kernel of eight rows at a time, in f16 times 2^15: 2^-11 size, and 2^-25 * 2^-15 of the row's largest;
    q there is f16 too, at least 224 at its largest: 2^-32 max|q|);
  - a logit's error ds in powers of two moves the output by 2 ln 2 ds size: q as hi + lo, 2^-17 max|q|
    an element; fp32 sums of d products; ex2 and the fused steps;
  - sums over the tokens, sixteen at least to a step: L / 16 * 2^-23, doubled."""
import math

import pytest
import torch

from hybrid_linear_attention_conv_gb300 import gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from hybrid_linear_attention_conv_gb300 import build
    build.build()
    gdn.load()
    assert torch.cuda.is_available()


def nearest(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


class Tail:
    """One request of L tokens, `new` of them queries, one key/value head; logits of all but
    token `at` are of order one."""

    def __init__(self, L, new, G, d, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.L, self.n, self.G, self.d = L, new, G, d
        pages = -(-L // PAGE)
        self.order = torch.randperm(pages, generator=g, device=DEV)
        k = torch.randn((pages * PAGE, d), generator=g, device=DEV) * 100
        k[:, 0] = 0
        v = torch.randn(d, generator=g, device=DEV) * 60 + torch.randn((pages * PAGE, d), generator=g, device=DEV) * 30
        self.k, self.v = nearest(k), nearest(v)
        self.ks = torch.full((pages,), 2.0 ** -7, device=DEV)
        self.vs = torch.full((pages,), 2.0 ** -6, device=DEV)
        self.q = torch.randn((new, G, d), generator=g, device=DEV).to(torch.bfloat16)
        self.q[..., 0] = 1.0

    def lift(self, at, bits):
        """Token `at`'s logits `bits` powers of two above (or below) what they are."""
        want = bits / (d_scale(self.d) * float(self.ks[at // PAGE]) * 448.0)
        self.k[at, 0] = math.copysign(448.0, want)
        self.q[..., 0] = abs(want)

    def share(self, at, part):
        """Token `at` with about that part of the last row's softmax."""
        others = torch.logsumexp(self.logits().masked_fill(torch.arange(self.L, device=DEV) == at, -math.inf)[-1, 0], 0) / math.log(2)
        self.lift(at, float(others) + math.log2(part / (1 - part)) - float(self.logits()[-1, 0, at]) / math.log(2))

    def logits(self):
        k = self.k.double() * self.ks.double().repeat_interleave(PAGE)[:, None]
        return torch.einsum("ngd,ld->ngl", self.q.double(), k[:self.L]) * self.d ** -0.5

    def run(self, tiles, copies=1):
        """copies: that many requests alike, over the same pages; the last one's rows are returned."""
        d, pages = self.d, self.ks.numel()
        codes = [torch.empty((pages, 1, PAGE, d), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
        scales = [torch.empty((pages, 1), device=DEV) for _ in range(2)]
        for c, s, x, y in zip(codes, scales, (self.k, self.v), (self.ks, self.vs)):
            c.view(torch.uint8)[self.order, 0] = x.view(torch.uint8).view(pages, PAGE, d)
            s[self.order, 0] = y
        # the kernel follows from the rows and the table's width: rows that no request has, and entries that none holds
        pad, width = (9, pages + ((1 << 22) + 8192) // PAGE) if tiles else (0, pages)
        table = torch.full((copies, width), -1, dtype=torch.int32, device=DEV)
        table[:, :pages] = self.order
        q = torch.cat([self.q.repeat(copies, 1, 1), self.q.new_zeros((pad, self.G, d))])
        i32 = dict(dtype=torch.int32, device=DEV)
        lse = torch.empty(q.shape[:2], device=DEV)
        out = gdn.kv_attention(q, *codes, *scales, table, torch.arange(copies + 1, **i32) * self.n, torch.full((copies,), self.L, **i32), lse=lse)
        last = slice((copies - 1) * self.n, copies * self.n)
        return out[last].double(), lse[last].double()

    def check(self, tiles, f16=False, copies=1, exact_q=False):
        """f16: the bound of the kernel of eight rows at a time; exact_q: no element of q is rounded."""
        out, lse = self.run(tiles, copies)
        L, d = self.L, self.d
        a, b = (s.double().repeat_interleave(PAGE)[:L] for s in (self.ks, self.vs))
        k, v = self.k.double()[:L], self.v.double()[:L]
        raw = torch.einsum("ngd,ld->ngl", self.q.double(), k) * a
        seen = torch.arange(L, device=DEV)[None] <= torch.arange(L - self.n, L, device=DEV)[:, None]
        s = (raw * d_scale(d)).masked_fill(~seen[:, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        w = torch.exp2(s - m)
        total = w.sum(-1, keepdim=True)
        w = w / total * b                                       # per code
        o, size = w @ v, w @ v.abs()
        blocks = torch.nn.functional.pad(w, (0, -L % 32)).unflatten(-1, (-1, 32))
        top = blocks.amax(-1, keepdim=True).expand_as(blocks).flatten(-2)[..., :L] * seen[:, None]
        q = self.q.double()
        ds = d_scale(d) * a * (q.abs().amax(-1, keepdim=True) * (0.0 if exact_q else 2.0 ** (-32 if f16 else -17)) * k.abs().sum(-1) + d * 2.0 ** -23 * (q.abs() @ k.abs().T))
        ds = (ds + 2.0 ** -21 + (s + b.log2()).abs() * 2.0 ** -22).masked_fill(~seen[:, None], 0)
        moved = 2 * math.log(2) * ds.amax(-1, keepdim=True)
        sums = L / 16 * 2.0 ** -22
        if f16:
            top = w.amax(-1, keepdim=True) * seen[:, None]
        held, below = (2.0 ** -11, 2.0 ** -40) if f16 else (2.0 ** -8 + 2.0 ** -12, 2.0 ** -22)
        bound = 2.0 ** -8 * o.abs() + (held + moved + sums) * size + below * (top @ v.abs())
        err = (out - o).abs()
        assert torch.isfinite(out).all()
        worst = float((err / bound).max())
        norm = float((err.norm(dim=-1) / (o.norm(dim=-1) + size.norm(dim=-1))).max())
        want = ((m + total.log2()) * math.log(2))[..., 0]
        lse_err = float(((lse - want).abs() / (moved[..., 0] + sums + want.abs() * 2.0 ** -22 + 2.0 ** -20)).max())
        print(f"L {L} d {d} tiles {tiles}: {worst:.3f} of the bound, {norm:.2e} of |o| + |size|, lse {lse_err:.3f}")
        assert worst <= 1 and lse_err <= 1
        # and as a whole: two roundings of 2^-8 to nearest, and the logits' part
        assert norm <= 2.0 ** -8 + float(moved.max()) + sums


def d_scale(d):
    return d ** -0.5 * math.log2(math.e)


FORMS = [(1, 6, 256), (130, 3, 256), (1, 8, 128), (130, 4, 128)]  # queries, rows a query, head size


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("new,G,d", FORMS)
@pytest.mark.parametrize("L,part", [(2048, 0.5), (2048, 0.95), (8192, 0.8), (8192, 0.9), (32768, 0.5), (32768, 0.95)])
def test_one_token_holds_much_of_the_softmax(L, part, new, G, d, tiles):
    t = Tail(L, new, G, d, seed=L)
    t.v[0] = nearest(t.v[0].float() * 0.01)  # a sink: its own value is small
    t.share(0, part)
    t.check(tiles)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("new,G,d", FORMS)
@pytest.mark.parametrize("L,at,bits", [(8192, 0, 10), (8192, 0, 14), (8192, 4099, 16), (8192, 0, 18), (8192, 5, 20), (30000, 0, 18),
                                       (30000, 29000, 16), (700, 0, 17)])
def test_a_token_without_value_far_above_the_rest(L, at, bits, new, G, d, tiles):
    t = Tail(L, new, G, d, seed=L + bits)
    t.v[at] = 0
    t.lift(at, bits)
    t.check(tiles)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("new,G,d", FORMS)
@pytest.mark.parametrize("bits", [8, 12, 14, 20])
def test_one_page_with_a_much_larger_value_scale(bits, new, G, d, tiles):
    """The page's scale comes from one token that is hardly attended to; its other tokens'
    codes are what is left of ordinary values."""
    L, page, at = 4096, 17, 17 * PAGE + 40
    t = Tail(L, new, G, d, seed=bits)
    t.vs[page] = 2.0 ** (bits - 6)
    rows = slice(page * PAGE, (page + 1) * PAGE)
    t.v[rows] = nearest(t.v[rows].float() * 2.0 ** -bits)
    t.v[at] = nearest(torch.randn(d, device=DEV) * 100)
    t.lift(at, -bits - 8.0)
    t.check(tiles)


@pytest.mark.parametrize("G,d", [(6, 256), (8, 128)])
@pytest.mark.parametrize("bits", [24, 30, 34, 36])
def test_eight_rows_keep_a_tail_far_below(bits, G, d):
    """One token a request, which is the kernel of eight rows whatever the table's width; so many
    requests that one is not spread over CTAs, whose parts have maxima of their own."""
    t = Tail(4096, 1, G, d, seed=bits)
    t.v[0] = 0
    t.lift(0, bits)
    t.check(False, f16=True, copies=1000)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("new,G,d", FORMS)
@pytest.mark.parametrize("large", [2.0 ** 8, 2.0 ** 12])
def test_a_query_with_one_large_channel(large, new, G, d, tiles):
    """Every other element of q is within 2^-14 of the large one, where q is exact: a channel
    whose keys are zero changes nothing, however large."""
    t = Tail(300, new, G, d, seed=int(large))
    g = torch.Generator(device=DEV).manual_seed(3)
    size = 0.5 + 1.5 * torch.rand((new, G, d), generator=g, device=DEV)
    t.q = (size * torch.sign(t.q.float())).to(torch.bfloat16)
    t.q[..., 0] = large
    t.ks.fill_(2.0 ** -5)  # peaked: logits of some units
    t.check(tiles, exact_q=True)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("new,G,d", FORMS)
@pytest.mark.parametrize("lo,hi", [(-40, 40), (-100, 10), (0, 110)])
def test_value_scales_far_apart(lo, hi, new, G, d, tiles):
    """Every page with a value scale of its own: the pages of the largest make the output, all
    of them the sum."""
    L = 3000
    t = Tail(L, new, G, d, seed=hi)
    g = torch.Generator(device=DEV).manual_seed(hi)
    t.vs = torch.exp2(torch.randint(lo, hi + 1, t.vs.shape, generator=g, device=DEV).float())
    t.vs[0], t.vs[1], t.vs[-1] = 2.0 ** lo, 2.0 ** hi, 2.0 ** lo
    t.check(tiles)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("new,G,d", FORMS)
@pytest.mark.parametrize("bits,seed", [(12, 0), (60, 1), (300, 2), (300, 3)])
def test_logits_that_jump_from_tile_to_tile(bits, seed, new, G, d, tiles):
    """Stretches of 32 to 256 tokens whose logits lie up to `bits` powers of two apart, up and down."""
    L = 5000
    t = Tail(L, new, G, d, seed=seed)
    g = torch.Generator().manual_seed(seed)
    level, i = torch.zeros(t.k.shape[0]), 0
    while i < L:
        n = 32 * int(torch.randint(1, 9, (), generator=g))
        level[i:i + n] = float(torch.randint(-448, 449, (), generator=g))
        i += n
    t.k[:, 0] = nearest(level).to(DEV)
    t.q[..., 0] = bits / 2 / (d_scale(d) * 2.0 ** -7 * 448.0)
    t.check(tiles)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("L,new", [(1, 1), (2, 2), (33, 33), (127, 3), (129, 129), (200, 1)])
@pytest.mark.parametrize("G,d", [(6, 256), (5, 128)])
def test_short_requests(L, new, G, d, tiles):
    t = Tail(L, new, G, d, seed=L)
    t.check(tiles)
