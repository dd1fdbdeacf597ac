"""Latent attention under wait limits between none and enough, with several blocks or items to a CTA, so that
waits give up anywhere in a CTA's list: every call ends, what it may not write stays as it was, a call that tells of nothing
is right, and so is whatever runs after it."""
import pytest
import torch

from hybrid_linear_attention_conv_gb300 import gdn
from latent_testutil import DEV, i32, starts
from test_gpu_latent import SCALE, expanded_case, latent_case

pytestmark = pytest.mark.gpu
LIMITS = [0] + [int(300 * 1.22 ** i) for i in range(28)]  # ns, up to about 65 us
EDGE = 4096                                               # elements on either side of an output


@pytest.fixture(scope="module", autouse=True)
def _built():
    from hybrid_linear_attention_conv_gb300 import build
    build.build()
    gdn.load()


class Inside:
    """Outputs within larger buffers of 7, of which rows `first` .. `last` - 1 may be written."""

    def __init__(self, T, H, d, first, last):
        self.buffers, self.views, self.rows = [], [], (first, last)
        for dtype, width in ((torch.bfloat16, H * d), (torch.float32, H)):
            buffer = torch.full((2 * EDGE + T * width,), 7.0, dtype=dtype, device=DEV)
            self.buffers.append(buffer)
            self.views.append(buffer[EDGE:EDGE + T * width].view(T, H, d) if dtype == torch.bfloat16 else buffer[EDGE:EDGE + T * width].view(T, H))

    def untouched(self):
        first, last = self.rows
        return all(bool((b[:EDGE] == 7).all() and (b[-EDGE:] == 7).all() and (v[:first] == 7).all() and (v[last:] == 7).all())
                   for b, v in zip(self.buffers, self.views))

    def refill(self):
        for b in self.buffers:
            b.fill_(7.0)


def under_limits(call, inside, want, after):
    """call(out, lse) under each limit; after() is a call of another kernel, which has to be right then."""
    gdn.kv_attention_status()
    assert gdn.kv_attention_status() == 0
    told = 0
    for limit in LIMITS:
        for _ in range(3):
            inside.refill()
            prev = gdn.set_wait_limit_ns(limit)
            try:
                call(*inside.views)
            finally:
                gdn.set_wait_limit_ns(prev)
            after()
            torch.cuda.synchronize()
            bad = gdn.kv_attention_status()
            told += bad != 0
            assert inside.untouched(), limit
            first, last = inside.rows
            assert bad or all(torch.equal(v[first:last], w) for v, w in zip(inside.views, want)), limit
    assert told >= 3  # those of a limit of 0 at least
    inside.refill()
    call(*inside.views)
    first, last = inside.rows
    assert all(torch.equal(v[first:last], w) for v, w in zip(inside.views, want)) and inside.untouched()
    assert gdn.kv_attention_status() == 0


def sentinel():
    """Another kernel's call with a status word of its own, checked."""
    c = latent_case(21, 16, 64, [300, 70], [1, 2])
    ws = torch.zeros(gdn.latent_attention_workspace_bytes(), dtype=torch.uint8, device=DEV)
    args = (c["q"], c["q_rope"], c["cache"], c["table"], c["start"], c["lens"], SCALE)
    want = gdn.latent_attention(*args, workspace=ws).clone()

    def after():
        assert torch.equal(gdn.latent_attention(*args, workspace=ws), want) and gdn.kv_attention_status(ws) == 0
    return after


# blocks of one tile, of two and three, of one and of two tiles of queries, with and without contexts; several to a CTA
@pytest.mark.parametrize("H,lens,new", [(32, [100] * 40, [100] * 40), (16, [300, 130, 20] * 14, [1, 130, 20] * 14), (24, [256] * 20, [256] * 20),
                                        (8, [390] * 90, [200] * 90)],
                         ids=["one tile", "chunks and single tokens", "two tiles of queries", "after contexts"])
def test_expanded_writes_nothing_outside(H, lens, new):
    c = expanded_case(22, H, lens, new)
    T, S, first = sum(new), sum(lens), 5
    q = torch.cat([c["q"][:first], c["q"], c["q"][:3]])  # rows of no request on either side
    start = i32([first + x for x in starts(new)])

    def call(out, lse):
        gdn.latent_attention_expanded(q, c["k"], c["k_rope"], c["v"], start, c["key_start"], SCALE, out=out, lse=lse)

    inside = Inside(T + first + 3, H, 128, first, first + T)
    call(*inside.views)
    want = [v[first:first + T].clone() for v in inside.views]
    under_limits(call, inside, want, sentinel())


@pytest.mark.parametrize("H,lens,new", [(160, [3000], [100]), (152, [128 * 5], [128]), (32, [2000] * 5, [3] * 5)],
                         ids=["joined", "five tiles", "few queries"])
def test_expanded_last_blocks_copies_land(H, lens, new):
    """A block or two to a CTA, whose loader is through with its copies long before they are used: a wait that gives up then
    must not end the CTA before they have landed (in what may be another's shared memory by then)."""
    c = expanded_case(23, H, lens, new)
    T = sum(new)

    def call(out, lse):
        gdn.latent_attention_expanded(c["q"], c["k"], c["k_rope"], c["v"], c["start"], c["key_start"], SCALE, out=out, lse=lse)

    inside = Inside(T, H, 128, 0, T)
    call(*inside.views)
    want = [v.clone() for v in inside.views]
    under_limits(call, inside, want, sentinel())


# items of 16, 32 and 64 rows, several to a CTA, of one tile and of many, whole and in parts; causal and by tree
@pytest.mark.parametrize("H,lens,new", [(8, [100] * 700, [1] * 700), (64, [200, 30] * 60, [1, 2] * 60), (128, [700] * 30, [1] * 30),
                                        (20, [3000, 64, 500] * 20, [1, 1, 3] * 20), (64, [300] * 8, [40] * 8)],
                         ids=["many short", "64 rows", "pairs", "parts", "chunks"])
def test_absorbed_ends_and_writes_nothing_outside(H, lens, new):
    c = latent_case(24, H, 64, lens, new)
    T, first = sum(new), 3
    q, r = (torch.cat([x[:first], x, x[:2]]) for x in (c["q"], c["q_rope"]))
    start = i32([first + x for x in starts(new)])
    ws = torch.zeros(gdn.latent_attention_workspace_bytes(), dtype=torch.uint8, device=DEV)

    def call(out, lse):
        gdn.latent_attention(q, r, c["cache"], c["table"], start, c["lens"], SCALE, out=out, lse=lse, workspace=ws)

    inside = Inside(T + first + 2, H, 512, first, first + T)
    call(*inside.views)
    want = [v[first:first + T].clone() for v in inside.views]
    under_limits(call, inside, want, sentinel())
