"""Sizes next to 2^31 are refused by the paged cache's calls: their kernels step through rows, pages and
tokens in 32 bits, past the last by a grid's stride or some tiles.

Every call's arguments fail validation, so no kernel is launched."""
import ctypes

import pytest

from hybrid_linear_attention_conv_gb300 import build as gbuild
from hybrid_linear_attention_conv_gb300 import gdn

P = ctypes.c_void_p
A, O, MOST = 0x10000, 0x20000, 0x7FF00000


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def shape(**kw):
    f = dict(B=2, Hq=8, Hkv=8, d=128, page=32, pages=100, width=10) | kw
    return ctypes.byref(gdn.gdn_kv_shape(*[f[k] for k, _ in gdn.gdn_kv_shape._fields_]))


def plan(lib, rows=4, cap=4, **kw):
    return lib.gdn_kv_plan(shape(**kw), P(A), P(A), P(A), P(A), cap, P(A), P(A), rows, P(O), P(O), P(O), P(O), P(O), P(O), None)


def attend(lib, T=4, **kw):
    return lib.gdn_kv_attention(shape(**kw), T, P(A), 8 * 128, P(A), P(A), P(A), P(A), P(A), P(A), P(A), None, 0.1, P(A), None, P(A),
                                1 << 30, None)


@pytest.mark.parametrize("n", [MOST + 1, 0x7FFFFFFF])
def test_rows_and_pages(lib, n):
    assert plan(lib, rows=n) == -2 and gdn.last_error()
    assert plan(lib, cap=n) == -2
    assert lib.gdn_kv_append(shape(), n, P(A), 1024, P(A), 1024, 4, P(A), P(A), P(A), P(A), P(A), P(A), None) == -2
    assert attend(lib, T=n) == -2
    assert attend(lib, T=n // 8 + 1, Hkv=1) == -2  # times eight heads of a group


@pytest.mark.parametrize("page", [32, 64, 128])
def test_tokens_of_a_table_row(lib, page):
    for width in (MOST // page + 1, 0x7FFFFFFF // page):
        assert plan(lib, page=page, width=width) == -2 and "tokens" in gdn.last_error()
        assert attend(lib, page=page, width=width) == -2 and "tokens" in gdn.last_error()
