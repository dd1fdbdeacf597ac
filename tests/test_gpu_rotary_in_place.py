"""Rotary positions in place: channels past the rotated ones are neither read nor written where their side has no norm, whatever
the other side does.  NaNs whose bits no conversion keeps lie there and show it; in the rotated channels and on the
other side everything is as it is out of place."""
import pytest
import torch

from hybrid_linear_attention_conv_gb300 import gdn
from latent_testutil import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from hybrid_linear_attention_conv_gb300 import build
    build.build()
    gdn.load()


@pytest.mark.parametrize("side", ["q", "k"])
@pytest.mark.parametrize("other", ["apart", "normed", "apart and normed", "in place"])
@pytest.mark.parametrize("T,Hq,Hk,d,rot,interleaved,dtype", [(1, 24, 4, 256, 64, False, torch.bfloat16), (300, 3, 5, 128, 96, True, torch.bfloat16),
                                                             (70, 8, 1, 64, 32, False, torch.float32), (9, 5, 2, 192, 16, False, torch.bfloat16)])
def test_channels_past_the_rotated_ones(side, other, T, Hq, Hk, d, rot, interleaved, dtype):
    g = torch.Generator(device=DEV).manual_seed(d)
    x = dict(q=torch.randn((T, Hq, d), generator=g, device=DEV).to(dtype), k=torch.randn((T, Hk, d), generator=g, device=DEV).to(dtype))
    away = "k" if side == "q" else "q"
    word, bits = (torch.int16, 0x7f85) if dtype == torch.bfloat16 else (torch.int32, 0x7f800123)
    positions = torch.randint(0, 5000, (T,), generator=g, device=DEV, dtype=torch.int32)
    turns, _ = gdn.rotary_frequencies(rot)
    norm = {away: 1 + 0.3 * torch.randn(d, generator=g, device=DEV) if "normed" in other else None, side: None}
    want = dict(zip("qk", gdn.rotary(x["q"], positions, turns, k=x["k"], q_norm=norm["q"], k_norm=norm["k"], interleaved=interleaved)))
    x[side].view(word)[:, :, rot:] = bits  # signalling NaNs
    out = {side: x[side], away: x[away] if "apart" not in other else torch.empty_like(x[away])}
    gdn.rotary(x["q"], positions, turns, k=x["k"], q_norm=norm["q"], k_norm=norm["k"], interleaved=interleaved, q_out=out["q"], k_out=out["k"])
    assert (x[side].view(word)[:, :, rot:] == bits).all()
    assert torch.equal(x[side][:, :, :rot], want[side][:, :, :rot])
    assert torch.equal(out[away], want[away])
