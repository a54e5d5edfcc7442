"""Host side of the cache's further calls: geometry of 4-bit pools, structures, refusals (no GPU)."""
import subprocess

import numpy as np
import pytest

import cache_more_ref as ref
import cache_ref
from prefill_decode_paged_gb300 import build as kbuild
from prefill_decode_paged_gb300 import kv_cache as kc
from prefill_decode_paged_gb300 import kv_relayout as kr
from test_host_cache import status

GOOD = dict(num_layers=2, num_components=2, kv_heads=8, head_dim=128, block=16, num_blocks=9, dtype=5, query_heads=32,
            max_requests=4, max_new=2)


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


@pytest.mark.parametrize("change, expected", [
    ({}, "KVR_OK"), (dict(head_dim=64), "KVR_OK"), (dict(head_dim=192), "KVR_OK"), (dict(head_dim=256), "KVR_OK"),
    (dict(head_dim=32), "KVR_ERR_UNSUPPORTED"), (dict(head_dim=96), "KVR_ERR_UNSUPPORTED"),
    (dict(head_dim=320), "KVR_ERR_UNSUPPORTED"),
    (dict(num_components=1, kv_heads=1, head_dim=576), "KVR_ERR_UNSUPPORTED"),
    (dict(num_components=1, kv_heads=1, head_dim=576, query_heads=0), "KVR_ERR_UNSUPPORTED"),
    (dict(scales=np.ones((2, 2))), "KVR_OK"), (dict(scales=np.ones((2, 2, 8)), per_head=True), "KVR_OK"),
    (dict(scales=np.array([[1, 0], [1, 1]])), "KVR_ERR_INVALID_ARG"),
    (dict(scales=np.array([[1, np.nan], [1, 1]])), "KVR_ERR_INVALID_ARG"),
    (dict(pool=None), "KVR_ERR_INVALID_ARG"), (dict(pool=(1 << 40) + 8), "KVR_ERR_ALIGNMENT"),
    (dict(pool=(1 << 64) - (1 << 16)), "KVR_ERR_UNSUPPORTED"), (dict(dtype=4), "KVR_ERR_UNSUPPORTED"),
    (dict(dtype=6), "KVR_ERR_UNSUPPORTED"),
])
def test_four_bit_geometry(change, expected):
    assert status(kc.workspace_bytes, 152, **dict(GOOD, **change)) == expected


def _layout(**change):
    lay = dict(bases=[(1 << 40) + i * (1 << 20) for i in range(4)], block_stride=16 * 8 * 64, token_stride=8 * 64,
               head_stride=64)
    return dict(lay, **change)


SCALES = [(1 << 41) + i * (1 << 20) for i in range(4)]


@pytest.mark.parametrize("change, scales, kw, expected", [
    ({}, SCALES, {}, "KVR_OK"),
    (dict(token_stride=64, head_stride=16 * 64), SCALES, {}, "KVR_OK"),
    (dict(token_stride=8 * 64 + 32), SCALES, {}, "KVR_ERR_ALIGNMENT"),       # scales' rows are read 8 bytes at a time
    (dict(token_stride=16 * 8 * 32 + 32, head_stride=96 * 2), SCALES, dict(head_dim=192, block=1), "KVR_OK"),
    (dict(token_stride=8 * 64 + 16), SCALES, dict(head_dim=64), "KVR_ERR_ALIGNMENT"),
    (dict(head_stride=0), SCALES, {}, "KVR_ERR_POOL_OVERLAP"),
    ({}, SCALES[:3] + [0], {}, "KVR_ERR_INVALID_ARG"),
    ({}, SCALES[:3] + [(1 << 42) + 8], {}, "KVR_ERR_ALIGNMENT"),
    ({}, SCALES[:3] + [(1 << 64) - 64], {}, "KVR_ERR_UNSUPPORTED"),
])
def test_four_bit_layouts(change, scales, kw, expected):
    assert status(kc.workspace_bytes, 152, layout=_layout(**change), block_scales=scales, **dict(GOOD, **kw)) == expected


def test_python_refuses_four_bit_pools_that_the_geometry_does_not_fit():
    import torch
    rows = 2 * 2 * 9 * 16 * 8
    pool = torch.zeros(rows * 72 - 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="holds"):
        kc.KVCache(pool, **GOOD)
    codes = [[[torch.zeros((9, 16, 8, 64), dtype=torch.uint8) for c in range(2)] for layer in range(2)]]
    lay = kr.layout_of_views(codes)
    good = [torch.zeros((9, 16, 8, 8), dtype=torch.uint8) for _ in range(4)]
    with pytest.raises(ValueError, match="block scales"):
        kc.KVCache(None, layout=lay, **GOOD)
    with pytest.raises(ValueError, match="block scales"):
        kc.KVCache(pool, block_scales=good, **GOOD)
    with pytest.raises(ValueError, match="block scales"):
        kc.KVCache(None, layout=lay, block_scales=good[:3], **GOOD)
    for bad in (good[0][:8], good[0][..., :4], good[0].transpose(1, 2).contiguous().transpose(1, 2),
                good[0].view(torch.int8).to(torch.int16)):
        with pytest.raises(ValueError, match="an eighth"):
            kc.KVCache(None, layout=lay, block_scales=good[:3] + [bad], **GOOD)
    if not torch.cuda.is_available():
        whole = torch.zeros(rows * 72, dtype=torch.uint8)
        assert status(kc.KVCache, whole, **GOOD) in ("KVR_ERR_CUDA", "KVR_ERR_POOL_ADDRESS")
        assert status(kc.KVCache, None, layout=lay, block_scales=good, **GOOD) in ("KVR_ERR_CUDA",
                                                                                   "KVR_ERR_POOL_ADDRESS")


def test_null_handles():
    lib = kc._library()
    buf = bytes(256)
    assert kr.STATUS[lib.kv_cache_append_at(None, 0, buf, None, None)] == "KVR_ERR_INVALID_ARG"
    assert kr.STATUS[lib.kv_cache_attend_scored(None, 0, buf, buf, None)] == "KVR_ERR_INVALID_ARG"
    assert kr.STATUS[lib.kv_cache_attend_scored(None, 0, buf, None, None)] == "KVR_ERR_INVALID_ARG"
    assert kr.STATUS[lib.kv_cache_weigh(None, 0, buf, None)] == "KVR_ERR_INVALID_ARG"
    assert kr.STATUS[lib.kv_cache_evict(None, 0, buf, None)] == "KVR_ERR_INVALID_ARG"
    assert kr.STATUS[lib.kv_cache_read(None, 0, buf, None)] == "KVR_ERR_INVALID_ARG"


def _offsets(tmp_path, expressions):
    """What these C expressions are, by the header."""
    src, exe = tmp_path / "s.c", tmp_path / "s"
    prints = "".join(f'    printf("%zu\\n", (size_t)({e}));\n' for e in expressions)
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kv_cache.h"\n'
                   f"int main(void) {{\n{prints}    return 0;\n}}\n")
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", kbuild.INCLUDE, str(src), "-o",
                    str(exe)], check=True)
    return [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]


def _marked(packed, field):
    """Where field number `field` of a packed structure begins."""
    n = len(packed.unpack(bytes(packed.size)))
    values = [0] * n
    values[field] = 0x1122
    return packed.pack(*values).index(b"\x22\x11")


def test_read_is_laid_out_as_the_binding_packs_it(tmp_path):
    got = _offsets(tmp_path, ["sizeof(kvc_read)", "offsetof(kvc_read, table)", "offsetof(kvc_read, k)",
                              "offsetof(kvc_read, v_head_stride)", "KVC_DTYPE_E2M1"])
    assert got == [kc._READ.size, _marked(kc._READ, 4), _marked(kc._READ, 8), _marked(kc._READ, 13),
                   kc.DTYPE_FP4_E2M1]


def test_scoring_is_laid_out_as_the_binding_packs_it(tmp_path):
    got = _offsets(tmp_path, ["sizeof(kvc_scoring)", "offsetof(kvc_scoring, slopes)"])
    assert got == [kc._SCORING.size, _marked(kc._SCORING, 2)]


def test_weigh_is_laid_out_as_the_binding_packs_it(tmp_path):
    fields = {"add": 5, "lengths": 6, "q": 11, "lse": 12, "weights": 13, "q_head_stride": 16, "weights_head_stride": 18,
              "weights_width": 19, "scoring.slopes": 23}
    got = _offsets(tmp_path, ["sizeof(kvc_weigh)"] + [f"offsetof(kvc_weigh, {n})" for n in fields])
    assert got == [kc._WEIGH.size] + [_marked(kc._WEIGH, f) for f in fields.values()]


def test_evict_is_laid_out_as_the_binding_packs_it(tmp_path):
    fields = {"weights_width": 3, "lengths": 4, "into": 9, "weights": 13, "weights_out": 14, "kept": 15,
              "out_head_stride": 19, "reserved": 20}
    got = _offsets(tmp_path, ["sizeof(kvc_evict)"] + [f"offsetof(kvc_evict, {n})" for n in fields])
    assert got == [kc._EVICT.size] + [_marked(kc._EVICT, f) for f in fields.values()]


def test_the_references_own_four_bits():
    """The tests' 64-bit forms: the codes' numbers, ties to even, and values that are codes already stay."""
    grid = ref.decode_e2m1(np.arange(16))
    assert list(grid[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and (grid[8:] == -grid[:8]).all()
    pos = grid[:8]
    ties = (pos[:-1] + pos[1:]) / 2
    assert list(ref.nearest(ties, pos)) == [0, 2, 2, 4, 4, 6, 6]
    assert list(ref.nearest([100, 0, 5.01, 4.99], pos)) == [7, 0, 7, 6]
    rng = np.random.default_rng(0)
    scale = np.repeat(cache_ref.decode_e4m3(rng.integers(1, 0x7F, (50, 4))), 16, -1)
    x = rng.choice(grid, (50, 64)) * scale
    x[:, ::16] = 6 * scale[:, ::16]
    assert (ref.values(*ref.quantize(x)) == x).all()
