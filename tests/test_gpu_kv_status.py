"""Attention calls without a workspace of the caller's: a bounded device wait that gave up is
still told, by the device's word.  A wait limit of 0 makes waits for copies just requested give
up at their first empty probe; the copies still land before the kernels end."""
import pytest
import torch

from hybrid_linear_attention_conv_gb300 import gdn
from test_gpu_kv import Step

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from hybrid_linear_attention_conv_gb300 import build
    build.build()
    gdn.load()


@pytest.mark.parametrize("new,tiles", [(1, False), (100, True)])
def test_a_give_up_without_a_workspace_is_told(new, tiles):
    s = Step([200000], [new], 24, 4, 256, 64, seed=21)
    gdn.kv_attention_status()  # whatever earlier calls left
    assert gdn.kv_attention_status() == 0
    prev = gdn.set_wait_limit_ns(0)
    try:
        s.run(tiles=tiles)
    finally:
        gdn.set_wait_limit_ns(prev)
    assert gdn.kv_attention_status() != 0
    assert gdn.kv_attention_status() == 0  # the reading cleared it
    s.check(got=s.run(tiles=tiles))
    assert gdn.kv_attention_status() == 0


def test_a_give_up_with_a_workspace_is_told_by_both():
    s = Step([200000], [1], 24, 4, 256, 64, seed=22)
    ws = torch.zeros(gdn.kv_attention_workspace_bytes(24, 4, 256), dtype=torch.uint8, device=DEV)
    gdn.kv_attention_status()
    prev = gdn.set_wait_limit_ns(0)
    try:
        s.run(workspace=ws)
    finally:
        gdn.set_wait_limit_ns(prev)
    assert gdn.kv_attention_status(ws) != 0 and gdn.kv_attention_status() != 0
    assert gdn.kv_attention_status(ws) != 0  # a workspace's word stays until it is zeroed


def test_a_captured_call_without_a_workspace():
    """The graph's calls keep a workspace inside it; their word is the device's."""
    s = Step([200000], [1], 24, 4, 256, 64, seed=23)
    ref = gdn.kv_attention(s.q, *s.cache, s.table, s.start, s.lens)
    out = torch.empty_like(s.q)
    graphs = []
    for limit in (0, None):
        prev = gdn.set_wait_limit_ns(0) if limit == 0 else None
        try:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                gdn.kv_attention(s.q, *s.cache, s.table, s.start, s.lens, out=out)
        finally:
            if prev is not None:
                gdn.set_wait_limit_ns(prev)
        graphs.append(graph)
    gdn.kv_attention_status()
    graphs[0].replay()  # captured with the limit of 0
    assert gdn.kv_attention_status() != 0
    graphs[1].replay()
    assert gdn.kv_attention_status() == 0
    assert torch.equal(out, ref)


def test_a_workspace_whose_words_are_anything_but_the_status():
    """Only the status word needs the zeroes."""
    s = Step([3000, 40], [1, 40], 8, 2, 128, 64, seed=24)
    for tiles in (False, True):
        ws = torch.full((gdn.kv_attention_workspace_bytes(8, 2, 128),), 0xFF, dtype=torch.uint8, device=DEV)
        ws[:4] = 0
        s.check(got=s.run(workspace=ws, tiles=tiles))
        assert gdn.kv_attention_status(ws) == 0
