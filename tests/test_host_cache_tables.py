"""Block tables as the binding hands them to the C library: the view's own rows."""
import numpy as np
import pytest
import torch

from prefill_decode_paged_gb300 import kv_cache as kc


def described(t):
    """What :meth:`KVCache._table` makes of a tensor, for a cache on the tensor's device."""
    cache = kc.KVCache.__new__(kc.KVCache)
    cache._h, cache._i32, cache._index, cache._device = None, torch.int32, t.get_device(), t.device
    return cache._table(t)


BASE = torch.arange(240, dtype=torch.int32)
VIEWS = [BASE.view(12, 20), BASE.view(12, 20)[:, 3:9], BASE.view(12, 20)[::2, :7], BASE[:6].expand(5, 6),
         BASE.as_strided((7, 6), (2, 1)), BASE.as_strided((7, 6), (0, 1), 11), BASE.view(12, 20)[:, :1],
         BASE.view(12, 20)[:1, 2:5], BASE[5:6].expand(4, 1), BASE.view(12, 20)[:, :0], BASE[:0].view(0, 5)]


@pytest.mark.parametrize("view", range(len(VIEWS)))
def test_rows_are_read_where_the_view_has_them(view):
    t = VIEWS[view]
    address, stride, rows, width = described(t)
    assert (rows, width) == tuple(t.shape) and stride >= 0
    flat, at = BASE.numpy(), (address - BASE.data_ptr()) // 4
    got = np.array([[flat[at + r * stride + e] for e in range(width)] for r in range(rows)], dtype=np.int32)
    np.testing.assert_array_equal(got.reshape(rows, width), t.numpy())


@pytest.mark.parametrize("t", [BASE.view(12, 20).t(), BASE.view(12, 20)[:, ::2], BASE, BASE.view(12, 20).long()])
def test_tables_whose_rows_are_not_rows_are_refused(t):
    with pytest.raises(ValueError, match="block table"):
        described(t)
