"""The paged 8-bit cache's entry points, without a GPU: what they refuse, their
sizes, and (tests/kv_index_check.cu, compiled for the host) the index
arithmetic that their kernels take their addresses from, bad pages included.

Every call is made with arguments that fail validation or that there is
nothing to do for, so no kernel is launched."""
import ctypes
import os
import shutil
import subprocess

import pytest

from hybrid_linear_attention_conv_gb300 import build as gbuild
from hybrid_linear_attention_conv_gb300 import gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
FAKE, OTHER = 0x10000, 0x20000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def test_index_arithmetic_and_exponents(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "kv_index_check")
    r = subprocess.run([nvcc, "-std=c++17", "-O1", *gbuild.ARCH, "-I", gbuild.INCLUDE, "-I", gbuild.CSRC,
                        os.path.join(ROOT, "tests", "kv_index_check.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout[-2000:]


def _sh(**kw):
    f = dict(B=2, Hq=24, Hkv=4, d=256, page=64, pages=100, width=10)
    f.update(kw)
    return gdn.gdn_kv_shape(*[f[k] for k, _ in gdn.gdn_kv_shape._fields_])


BAD_SHAPES = [dict(d=64), dict(d=96), dict(page=16), dict(page=48), dict(page=256), dict(Hq=23), dict(Hkv=0), dict(Hq=0),
              dict(B=-1), dict(pages=-1), dict(width=-1), dict(Hq=2048), dict(pages=1 << 24)]


def _plan(lib, sh, lens=FAKE, add=FAKE, held=FAKE, free=FAKE, cap=4, count=FAKE, table=FAKE, rows=4, lens_out=OTHER,
          held_out=OTHER, count_out=OTHER, start=OTHER, slots=OTHER, status=OTHER):
    return lib.gdn_kv_plan(ctypes.byref(sh) if sh else None, P(lens), P(add), P(held), P(free), cap, P(count), P(table), rows,
                           P(lens_out), P(held_out), P(count_out), P(start), P(slots), P(status), None)


def _append(lib, sh, T=4, k=FAKE, ldk=1024, v=FAKE, ldv=1024, n=4, slots=FAKE, rows=None, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE):
    return lib.gdn_kv_append(ctypes.byref(sh) if sh else None, T, P(k), ldk, P(v), ldv, n, P(slots), P(rows), P(kc), P(vc), P(ks),
                             P(vs), None)


def _attend(lib, sh, T=4, q=FAKE, ldq=6144, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, start=FAKE, lens=FAKE, tree=None,
            scale=0.0625, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 30):
    return lib.gdn_kv_attention(ctypes.byref(sh) if sh else None, T, P(q), ldq, P(kc), P(vc), P(ks), P(vs), P(table), P(start),
                                P(lens), P(tree), scale, P(out), P(lse), P(ws), ws_bytes, None)


@pytest.mark.parametrize("bad", BAD_SHAPES, ids=str)
def test_bad_shapes_are_refused(lib, bad):
    sh = _sh(**bad)
    for call in (_plan, _append, _attend):
        assert call(lib, sh) == -2 and gdn.last_error()
    assert lib.gdn_kv_attention_workspace_bytes(ctypes.byref(sh)) == 0


def test_null_shape(lib):
    assert _plan(lib, None) == _append(lib, None) == _attend(lib, None) == -1


def test_plan_refusals(lib):
    assert _plan(lib, _sh(B=12289)) == -2
    assert _plan(lib, _sh(width=1 << 26)) == -2  # more tokens than 32 bits count
    assert _plan(lib, _sh(), rows=-1) == -1
    assert _plan(lib, _sh(), cap=-1) == -1
    for name in ("lens", "add", "held", "free", "count", "table", "lens_out", "held_out", "count_out", "start", "slots", "status"):
        assert _plan(lib, _sh(), **{name: None}) == -1, name
        assert _plan(lib, _sh(), **{name: FAKE + 4}) == -6, name
    assert _plan(lib, _sh(), lens_out=FAKE) == -1  # in place
    assert _plan(lib, _sh(), count_out=FAKE) == -1 and "distinct" in gdn.last_error()


def test_append_refusals(lib):
    assert _append(lib, _sh(), T=-1) == -1
    assert _append(lib, _sh(), n=-1) == -1
    assert _append(lib, _sh(), n=3) == -1           # fewer source rows than rows
    assert _append(lib, _sh(), ldk=1016) == -1      # below a row
    assert _append(lib, _sh(), ldv=1028) == -6      # not a multiple of 16 bytes
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert _append(lib, _sh(), **{name: None}) == -1, name
        assert _append(lib, _sh(), **{name: FAKE + 8}) == -6, name
    assert _append(lib, _sh(), rows=FAKE + 4) == -6
    assert _append(lib, _sh(), T=0, k=None, slots=None) == 0
    assert _append(lib, _sh(pages=0)) == 0


def test_attention_refusals(lib):
    assert _attend(lib, _sh(), T=-1) == -1
    assert _attend(lib, _sh(), ldq=6136) == -1
    assert _attend(lib, _sh(), ldq=6148) == -6
    for scale in (0.0, -1.0, float("nan"), float("inf"), 2e6):
        assert _attend(lib, _sh(), scale=scale) == -1, scale
    for name in ("q", "kc", "vc", "ks", "vs", "table", "start", "lens", "out"):
        assert _attend(lib, _sh(), **{name: None}) == -1, name
        assert _attend(lib, _sh(), **{name: FAKE + 8}) == -6, name
    assert _attend(lib, _sh(), tree=FAKE + 8) == -6
    assert _attend(lib, _sh(), lse=FAKE + 8) == -6
    assert _attend(lib, _sh(), ws=None) == -9
    assert _attend(lib, _sh(), ws=FAKE + 16) == -6
    need = lib.gdn_kv_attention_workspace_bytes(ctypes.byref(_sh()))
    assert need > 0 and _attend(lib, _sh(), ws_bytes=need - 1) == -9
    assert _attend(lib, _sh(pages=0)) == -2
    assert _attend(lib, _sh(width=0)) == -2
    assert _attend(lib, _sh(width=1 << 26)) == -2
    assert _attend(lib, _sh(), T=0, q=None) == 0
    assert _attend(lib, _sh(B=0), q=None) == 0


def test_status_reader_refuses_null(lib):
    assert lib.gdn_kv_attention_status(None, None, None) == -9


def test_python_checks():
    import torch
    t = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        gdn.kv_append(t, t, torch.zeros(4, dtype=torch.int64), *[torch.zeros((1, 8, 32, 128), dtype=torch.float8_e4m3fn)] * 2,
                      *[torch.zeros((1, 8))] * 2)
    with pytest.raises(ValueError):
        gdn.kv_append(t, t, torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.zeros(4), torch.zeros(4), torch.zeros(4))
