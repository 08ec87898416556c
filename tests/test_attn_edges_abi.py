"""Edges of the paged-cache entry points on the host (nothing valid enough to launch is
passed)."""
import pytest

from tests.test_attn_abi import FAKE, INVALID, SHAPE, WORKSPACE, L, append, attend  # noqa: F401

OK = 0


@pytest.mark.parametrize("page", [8, 64, 256])
def test_positions_leave_room_for_rounding_up(L, page):
    # a length of 2^31 - 8 rounded up to tiles of 128 keys would leave 32 bits
    for max_pages in ((2 ** 31 - 1) // page, (2 ** 31 - 1024) // page + 1):
        kw = dict(page_size=page, max_pages=max_pages)
        assert append(L, kw) == SHAPE
        assert attend(L, kw) == SHAPE
        assert attend(L, kw, prefix=(FAKE, FAKE, 1)) == SHAPE
    kw = dict(page_size=page, max_pages=(2 ** 31 - 1024) // page)
    assert append(L, kw, ws=None) == attend(L, kw, ws=None) == WORKSPACE


def test_calls_need_the_caches_device_to_be_current(L):
    kv = object.__new__(L.PagedKV)
    kv._device, kv._current_device = 1, lambda: 1
    kv._current_stream = lambda device: 100 + device
    assert kv.stream(None) == 101
    kv._current_device = lambda: 0
    with pytest.raises(ValueError, match="current device"):
        kv.stream(None)


def test_an_empty_batch_has_no_rows_to_point_to(L):
    none = dict(T=0)
    assert append(L, none, q=None, k=None, v=None, qo=None) == OK
    assert append(L, none, q=None, k=None, v=None, qo=None, axes=3, pairs=[8, 12, 12]) == OK
    assert append(L, none, q=None, k=None, v=None, qo=None, axes=3) == INVALID      # the pairs are host memory
    for prefix in (None, (FAKE, FAKE, 2)):
        assert attend(L, none, prefix=prefix, q=None, out=None) == OK
        assert attend(L, none, prefix=prefix, q=None, out=None, scale=0.0) == INVALID
        assert attend(L, prefix=prefix, q=None, out=None) == INVALID
        assert attend(L, none, prefix=prefix, q=FAKE, out=FAKE) == INVALID
