"""The absorbed form where a token's logits are all -inf but its values are finite: its weight is zero and it changes nothing,
wherever it lies in the context.  (In tiles that not every row sees, a row whose logits are all not finite used to be taken for
one whose values are not, and made NaN of the rows that see it.)

Tolerances are latent_testutil's for every element.  Its 2-norm's (0.004) is for softmaxes of many tokens, whose weights'
roundings are independent; with a query channel of 30 or more one token has nearly all of a row's, and the row's elements share that weight's
rounding: 2^-8 of the output, beside 2^-8 / sqrt 3 for the output's own: 0.0062 here."""
import math

import pytest
import torch

from hybrid_linear_attention_conv_gb300 import gdn
from latent_testutil import attend, seen_mask
from test_gpu_latent import ROOM, SCALE, latent_case, room, rows_of, run_latent  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from hybrid_linear_attention_conv_gb300 import build
    build.build()
    gdn.load()


def within(got, lse, want, want_lse, bound, lse_bound):
    got, lse = got.double(), lse.double()
    empty = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (got[empty] == 0).all()
    assert ((got - want).abs() <= bound).all() and ((lse - want_lse).abs()[~empty] <= lse_bound[~empty]).all()
    assert float((got - want).norm()) <= (2.0 ** -8 + 2.0 ** -8 / math.sqrt(3.0)) * float(want.norm())


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("kind", ["key part", "sum"])
@pytest.mark.parametrize("H,n,L,at", [(64, 1, 130, 129), (64, 1, 130, 10), (16, 1, 70, 64), (16, 1, 200, 3), (32, 1, 65, 64), (16, 4, 300, 297),
                                      (64, 3, 130, 128), (128, 2, 90, 88), (16, 8, 64, 60), (64, 2, 4000, 3998)])
def test_logits_of_minus_infinity(kind, H, n, L, at):
    c = latent_case(31, H, 64, [L, 70], [n, 1])
    row = c["cache"][c["table"][0, at // 64], at % 64]
    if kind == "key part":   # -inf times a positive number in every query
        c["q_rope"][:, :, 5] = c["q_rope"][:, :, 5].abs() + 0.5
        row[512 + 5] = -float("inf")
    else:                    # finite, but past fp32's range in every query's sum
        c["q"][:, :, 7] = c["q"][:, :, 7].abs() + 30
        row[7] = -3.0e38
    out, lse = run_latent(c)
    t = 0
    for b, (length, new) in enumerate(((L, n), (70, 1))):
        x = rows_of(c["cache"], c["table"], b, length).clone()
        seen = seen_mask(new, length)
        if b == 0:
            x[at] = 0
            seen[:, at] = False
        for h in range(H):
            q = torch.cat([c["q"][t:t + new, h], c["q_rope"][t:t + new, h]], -1)
            within(out[t:t + new, h], lse[t:t + new, h], *attend(q, x, x[:, :512], seen, SCALE))
        t += new


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("H,n,L,at", [(64, 1, 130, 129), (64, 1, 130, 10), (32, 2, 65, 64), (128, 2, 90, 88), (16, 130, 400, 300)])
def test_values_that_are_not_finite_reach_their_channels(H, n, L, at):
    """... and a value that is not finite still reaches every row that sees it, with a weight of zero too (0 times inf), and no other."""
    c = latent_case(32, H, 64, [L, 70], [n, 1])
    c["q"][:, :, 7] = c["q"][:, :, 7].abs() + 0.5
    want, want_lse = run_latent(c)
    c["cache"][c["table"][0, at // 64], at % 64, 7] = -float("inf")
    out, lse = run_latent(c)
    blind = max(0, at - (L - n))
    assert torch.equal(out[:blind], want[:blind]) and torch.equal(lse[:blind], want_lse[:blind]) and torch.equal(out[n:], want[n:])
    assert out[blind:n, :, 7].isnan().all()
