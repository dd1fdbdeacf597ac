"""Rows that are not finite and are taken back again, as a speculative round does with a rejected
draft: the cache is then what it would be without them, bit for bit."""
import math

import pytest
import torch

from hybrid_linear_attention_conv_gb300 import gdn
from test_gpu_kv import check_append, new_cache, rows_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from hybrid_linear_attention_conv_gb300 import build
    build.build()
    gdn.load()


def append(k, v, first, cache, page, rows=None):
    slots = torch.arange(first, first + (len(k) if rows is None else len(rows)), device=DEV)
    gdn.kv_append(k, v, slots, *cache, rows=None if rows is None else torch.tensor(rows, dtype=torch.int32, device=DEV))


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("bad", [math.nan, -math.inf])
@pytest.mark.parametrize("context,drafts,at,path", [(10, 9, 4, [0, 1, 2]), (10, 3, 0, [1, 2]), (1, 30, 29, range(29)), (20, 2, 1, [0]),
                                                    (27, 4, 2, [0, 1, 3]), (0, 12, 5, [0, 6, 11])])
def test_rejected_drafts_that_are_not_finite(context, drafts, at, path, bad, d, page):
    """Of `drafts` nodes those of `path` are accepted; number `at` is bad."""
    Hkv, first = 3, page  # the context begins page 1
    k, v = rows_of(64, Hkv, d, seed=context + at, spread=1.0)
    k, v = k.clone(), v.clone()
    small = slice(context, context + drafts)  # drafts within the context's scale, which they leave as it is
    if context:
        k[small] *= 2.0 ** -12
        v[small] *= 2.0 ** -12
    got, want = new_cache(4, Hkv, page, d), new_cache(4, Hkv, page, d)
    assert same(got, want)
    if context:
        append(k[:context], v[:context], first, got, page)
        append(k[:context], v[:context], first, want, page)
    dk, dv = k[small].clone(), v[small].clone()
    dk[at, 1, 7] = bad
    dv[at, 2, d - 1] = bad
    append(dk, dv, first + context, got, page)
    assert torch.isnan(got[2][1, 1]) and torch.isnan(got[3][1, 2]) and not torch.isnan(got[2][1, 0])
    codes = [c.float() for c in got[:2]]
    assert all(torch.isfinite(c[1]).all() for c in codes)
    # the accepted drafts again, gathered; in the other cache only they ever were
    path = list(path)
    append(dk, dv, first + context, got, page, rows=path)
    append(dk, dv, first + context, want, page, rows=path)
    end = context + len(path)
    for x, y in zip(got[:2], want[:2]):
        assert torch.equal(x.view(torch.uint8)[1, :, :end], y.view(torch.uint8)[1, :, :end])
    for x, y in zip(got[2:], want[2:]):
        assert torch.isfinite(x[1]).all() and torch.equal(x[1], y[1])


@pytest.mark.parametrize("n", [2, 20])
def test_a_row_that_stays_keeps_its_block_lost(n):
    page, d, Hkv = 64, 256, 2
    cache = new_cache(3, Hkv, page, d)
    k, v = rows_of(64, Hkv, d, seed=1)
    k = k.clone()
    k[5, 0, 0] = math.inf
    append(k[:10], v[:10], 64, cache, page)
    for first in (10, 6):  # after it, twice: the mark stays too
        append(k[20:20 + n], v[20:20 + n], 64 + first, cache, page)
        assert torch.isnan(cache[2][1, 0]) and not torch.isnan(cache[2][1, 1])
    append(k[20:20 + n], v[20:20 + n], 64 + 5, cache, page)
    assert torch.isfinite(cache[2][1, 0])


def test_a_scale_of_the_callers_that_is_no_power_of_two_is_lost():
    page, d, Hkv = 32, 128, 1
    cache = new_cache(2, Hkv, page, d)
    cache[2].fill_(0.75)
    cache[3].fill_(0.75)
    k, v = rows_of(8, Hkv, d, seed=2, spread=0.0)
    k = k.clone()
    k[1, 0, 0] = math.nan
    append(k[:2], v[:2], 8, cache, page)
    append(k[2:3], v[2:3], 9, cache, page)
    assert torch.isnan(cache[2][0, 0]) and cache[3][0, 0] == 0.75
    check_append(k[2:4], v[2:4], [0, 1], cache, page)  # begun again
