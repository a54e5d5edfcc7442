"""Host side of the decode cache: the C header, the binding's structures, refusals, rotation tables."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import cache_ref
from prefill_decode_paged_gb300 import KVRelayoutError, build as kbuild, rotary_table
from prefill_decode_paged_gb300 import kv_cache as kc
from prefill_decode_paged_gb300 import kv_relayout as kr

HEADER = os.path.join(kbuild.INCLUDE, "kv_cache.h")


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


def test_library_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(kv_cache_\w+)\s*\(", text))
    assert names == set(kc.CACHE_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", kr.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (kv_cache_\w+)", out))


def test_header_is_c99_and_structures_are_laid_out_as_the_binding_packs_them(tmp_path):
    code = """
#include <stddef.h>
#include <stdio.h>
#include "kv_cache.h"
int main(void) {
    printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu %zu %d\\n", sizeof(kvc_desc), sizeof(kvc_append),
           sizeof(kvc_attend), sizeof(kvc_scaling), offsetof(kvc_append, rotary),
           offsetof(kvc_append, q_out_head_stride), offsetof(kvc_attend, lse),
           offsetof(kvc_attend, out_head_stride), offsetof(kvc_desc, query_heads),
           offsetof(kvc_scaling, magnitude), KVC_MAX_REQUESTS);
    return 0;
}
"""
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text(code)
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                    kbuild.INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    a, t = kc._APPEND, kc._ATTEND
    assert got[:4] == [ctypes.sizeof(kc.KvcDesc), a.size, t.size, ctypes.sizeof(kc.KvcScaling)]
    # offsets: marks packed one by one land where C has them
    fields = [0] * 27
    assert len(a.unpack(bytes(a.size))) == len(fields)
    fields[14] = 0x1122
    assert a.pack(*fields).index(b"\x22\x11") == got[4]
    fields = [0] * 27
    fields[26] = 0x1122
    assert a.pack(*fields).index(b"\x22\x11") == got[5]
    n = len(t.unpack(bytes(t.size)))
    fields = [0] * n
    fields[13] = 0x1122
    assert t.pack(*fields).index(b"\x22\x11") == got[6]
    fields = [0] * n
    fields[n - 1] = 0x1122
    assert t.pack(*fields).index(b"\x22\x11") == got[7]
    assert got[8] == kc.KvcDesc.query_heads.offset and got[9] == kc.KvcScaling.magnitude.offset
    assert got[10] == 2048


GOOD = dict(num_layers=2, num_components=2, kv_heads=8, head_dim=128, block=16, num_blocks=9, dtype=1,
            query_heads=32, max_requests=4, max_new=2)


def status(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except KVRelayoutError as e:
        return e.name
    return "KVR_OK"


@pytest.mark.parametrize("change, expected", [
    ({}, "KVR_OK"),
    (dict(num_layers=0), "KVR_ERR_INVALID_ARG"),
    (dict(num_components=3), "KVR_ERR_INVALID_ARG"),
    (dict(kv_heads=0), "KVR_ERR_INVALID_ARG"),
    (dict(block=0), "KVR_ERR_INVALID_ARG"),
    (dict(num_blocks=0), "KVR_ERR_INVALID_ARG"),
    (dict(num_blocks=1 << 31), "KVR_ERR_UNSUPPORTED"),
    (dict(dtype=0), "KVR_ERR_UNSUPPORTED"),
    (dict(dtype=4), "KVR_ERR_UNSUPPORTED"),
    (dict(head_dim=24), "KVR_ERR_UNSUPPORTED"),
    (dict(head_dim=272), "KVR_ERR_UNSUPPORTED"),
    (dict(head_dim=256), "KVR_OK"),
    (dict(head_dim=16), "KVR_OK"),
    (dict(value_dim=64), "KVR_ERR_UNSUPPORTED"),
    (dict(query_heads=12), "KVR_ERR_INVALID_ARG"),
    (dict(query_heads=-8), "KVR_ERR_INVALID_ARG"),
    (dict(query_heads=0, max_requests=0), "KVR_OK"),
    (dict(max_requests=0), "KVR_ERR_INVALID_ARG"),
    (dict(max_requests=2049), "KVR_ERR_UNSUPPORTED"),
    (dict(max_new=0), "KVR_ERR_INVALID_ARG"),
    (dict(dtype=2), "KVR_ERR_INVALID_ARG"),                                  # no scales
    (dict(dtype=2, scales=np.ones((2, 2))), "KVR_OK"),
    (dict(dtype=2, scales=np.ones((2, 2, 8)), per_head=True), "KVR_OK"),
    (dict(dtype=2, scales=np.array([[1, 0], [1, 1]])), "KVR_ERR_INVALID_ARG"),
    (dict(dtype=2, scales=np.array([[1, np.inf], [1, 1]])), "KVR_ERR_INVALID_ARG"),
    (dict(scales=np.ones((2, 2))), "KVR_ERR_INVALID_ARG"),                   # not an E4M3 pool
    (dict(pool=None), "KVR_ERR_INVALID_ARG"),
    (dict(pool=(1 << 40) + 8), "KVR_ERR_ALIGNMENT"),
    (dict(num_components=1, kv_heads=1, head_dim=576), "KVR_OK"),
    (dict(num_components=1, kv_heads=1, head_dim=512), "KVR_ERR_UNSUPPORTED"),
    (dict(num_components=1, kv_heads=2, head_dim=576), "KVR_ERR_UNSUPPORTED"),
    (dict(num_components=1, kv_heads=1, head_dim=576, dtype=2, scales=np.ones((2, 1))),
     "KVR_ERR_UNSUPPORTED"),
    (dict(num_components=1, kv_heads=1, head_dim=576, dtype=2, scales=np.ones((2, 1)),
          query_heads=0), "KVR_OK"),
])
def test_geometry_refusals(change, expected):
    assert status(kc.workspace_bytes, 152, **dict(GOOD, **change)) == expected


def _layout(**change):
    row = 128 * 2
    lay = dict(bases=[(1 << 40) + i * (1 << 20) for i in range(4)], block_stride=16 * 8 * row,
               token_stride=8 * row, head_stride=row)
    return dict(lay, **change)


@pytest.mark.parametrize("change, expected", [
    ({}, "KVR_OK"),
    (dict(token_stride=128 * 2, head_stride=16 * 128 * 2), "KVR_OK"),        # head-major blocks
    (dict(token_stride=8 * 256 + 8), "KVR_ERR_ALIGNMENT"),
    (dict(head_stride=240), "KVR_ERR_POOL_OVERLAP"),
    (dict(token_stride=-16), "KVR_ERR_INVALID_ARG"),
    (dict(bases=[1 << 40, 0, 1 << 41, 1 << 42]), "KVR_ERR_INVALID_ARG"),
    (dict(bases=[1 << 40, (1 << 41) + 4, 1 << 42, 1 << 43]), "KVR_ERR_ALIGNMENT"),
    (dict(block_stride=1 << 62), "KVR_ERR_UNSUPPORTED"),
])
def test_layout_refusals(change, expected):
    assert status(kc.workspace_bytes, 152, layout=_layout(**change), **GOOD) == expected


def test_null_handles_and_out_arguments():
    lib = kc._library()
    buf = bytes(256)
    assert kr.STATUS[lib.kv_cache_append(None, 0, buf, None)] == "KVR_ERR_INVALID_ARG"
    assert kr.STATUS[lib.kv_cache_attend(None, 0, buf, None)] == "KVR_ERR_INVALID_ARG"
    assert kr.STATUS[lib.kv_cache_status(None, None)] == "KVR_ERR_INVALID_ARG"
    assert kr.STATUS[lib.kv_cache_create(None, None)] == "KVR_ERR_INVALID_ARG"
    h = ctypes.c_void_p(7)
    assert kr.STATUS[lib.kv_cache_create(None, ctypes.byref(h))] == "KVR_ERR_INVALID_ARG"
    assert h.value is None
    lib.kv_cache_destroy(None)


def test_python_refuses_pools_that_the_geometry_does_not_fit():
    import torch
    pool = torch.zeros((2, 2, 9, 16, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="holds"):
        kc.KVCache(pool[:1], **GOOD)
    with pytest.raises(ValueError, match="contiguous"):
        kc.KVCache(pool.transpose(0, 1), **GOOD)
    with pytest.raises(ValueError, match="scales"):
        kc.KVCache(pool.view(torch.uint8), **dict(GOOD, dtype=2), scales=np.ones(3))
    views = kr.layout_of_views([[[pool[l, c] for c in range(2)] for l in range(2)]])
    with pytest.raises(ValueError, match="addresses"):
        kc.KVCache(None, layout=views, **dict(GOOD, block=32))
    with pytest.raises(ValueError, match="views"):
        kc.KVCache(None, layout=views, **dict(GOOD, num_layers=1))
    if not torch.cuda.is_available():
        assert status(kc.KVCache, pool, **GOOD) in ("KVR_ERR_CUDA", "KVR_ERR_POOL_ADDRESS")


SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="base", factor=2.5),
            dict(kind="ramp", factor=8.0, original=4096),
            dict(kind="ramp", factor=40.0, original=4096, beta_fast=16.0, beta_slow=2.0, magnitude=1.25),
            dict(kind="bands", factor=8.0, original=8192, beta_fast=4.0, beta_slow=1.0)]


@pytest.mark.parametrize("dim", [16, 64, 128])
@pytest.mark.parametrize("scaling", SCALINGS)
def test_rotary_table_is_the_formula_rounded_once(dim, scaling):
    got = rotary_table(300, dim, 10000.0, scaling)
    ref = cache_ref.rotary_table(300, dim, 10000.0, scaling)
    # two fp64 evaluations of angles up to 300, and one rounding to fp32
    assert got.dtype == np.float32 and got.shape == (300, dim)
    np.testing.assert_allclose(got, ref, rtol=0, atol=2.0 ** -24 * 1.5 + 300 * 2.0 ** -50)


def test_rotary_table_at_far_positions():
    got = rotary_table(200000, 16, 500000.0)
    ref = cache_ref.rotary_table(200000, 16, 500000.0)
    np.testing.assert_allclose(got, ref, rtol=0, atol=2.0 ** -24 + 200000 * 2.0 ** -50)


@pytest.mark.parametrize("args, kw, error", [
    ((0, 64), {}, "KVR_ERR_INVALID_ARG"), ((4, 63), {}, "KVR_ERR_INVALID_ARG"),
    ((4, 64, 1.0), {}, "KVR_ERR_INVALID_ARG"),
    ((4, 64), dict(scaling=dict(kind="linear", factor=0.5)), "KVR_ERR_INVALID_ARG"),
    ((4, 64), dict(scaling=dict(kind="ramp", factor=2.0)), "KVR_ERR_INVALID_ARG"),
    ((4, 64), dict(scaling=dict(kind="bands", factor=2.0, original=8, beta_fast=1.0)),
     "KVR_ERR_INVALID_ARG"),
])
def test_rotary_table_refusals(args, kw, error):
    assert status(rotary_table, *args, **kw) == error


def test_rotary_table_refuses_unknown_scalings():
    with pytest.raises(ValueError):
        rotary_table(4, 64, scaling=dict(kind="other", factor=2.0))
    with pytest.raises(ValueError):
        rotary_table(4, 64, scaling=dict(kind="linear", factor=2.0, extra=1))


def test_reference_rotation_keeps_lengths_and_e4m3_grid_is_the_formats():
    """The tests' own 64-bit forms: a rotation keeps each pair's length, codes stand for what the
    format says."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 32))
    t = cache_ref.rotary_table(9, 32, 10000.0)
    for il in (False, True):
        y = cache_ref.rotate(x, [0, 3, 8, 1, -1], t, 32, il, False)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        np.testing.assert_array_equal(y[0], x[0])
        np.testing.assert_array_equal(y[4], x[4])
    g = cache_ref.e4m3_grid()
    assert len(g) == 253 and g[-1] == 448 and g[g > 0][0] == 2.0 ** -9
