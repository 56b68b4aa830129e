"""Sizes at the edge of 32 bits, without a GPU: what does not fit the C calls'
fields is refused or cut to them, never taken modulo 2^32."""
import ctypes

import pytest

from test_layer_checks import OK, _buf, _cfg, _create, _view, lib  # noqa: F401


@pytest.mark.parametrize("name, value", [
    ("heads", 2 ** 32 + 4), ("kv_heads", 2 ** 32 + 2), ("d", 2 ** 32 + 64), ("rope_orig", 2 ** 32 + 8),
    ("page_size", 2 ** 32 + 16), ("causal_block", 2 ** 32 + 1), ("window", 2 ** 32), ("window", 2 ** 31),
    ("window", -2 ** 32 + 5), ("rope_max", (2 ** 32 + 5, 7)), ("rope_dims", (2 ** 32 + 16, 24)),
])
def test_config_fields_past_32_bits(name, value):
    with pytest.raises(ValueError, match=name):
        _cfg(**{name: value})


def test_config_fields_that_fit(lib):
    got, h = _create(lib, window=2 ** 31 - 1, causal_block=2 ** 31 - 1)
    assert got == OK
    lib.ac_layer_destroy(h)


def test_call_bounds_past_32_bits():
    """max_q and max_kv are bounds: more than fits means no bound, less than 0 stays wrong."""
    from clustered_sparse_attention_head_b200.layer import _int32
    top = 2 ** 31 - 1
    for value, want in ((0, 0), (7, 7), (top, top), (2 ** 31, top), (2 ** 32, top), (2 ** 40 + 3, top), (-1, -1),
                        (-2 ** 31, -2 ** 31), (-2 ** 32 + 5, -2 ** 31)):
        assert _int32(value) == want


def test_longest_sequence(lib):
    """The keys of a call stay so far below 2^31 that a chunk's end, a page's and a
    tile's are still 32-bit numbers."""
    code, h = _create(lib)
    need = ctypes.c_size_t()
    lib.ac_layer_workspace_size(h, ctypes.byref(need))
    raw, base = _buf()
    q, out = _view(base, 0, 256, 64), _view(base + 8192, 0, 256, 64)
    for max_kv, max_pages in ((2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 27), (2 ** 31 - 100, 2 ** 28)):
        assert lib.ac_cache_attn(h, 2, 5, 5, max_kv, base, base, base, max_pages, 4, ctypes.byref(q), base, base,
                                 ctypes.byref(out), None, base, need.value, None) == OK
        assert lib.stub_attn(1) == 2 ** 31 - 2 ** 16
    assert lib.ac_cache_attn(h, 2, 5, 5, 2 ** 31 - 1, base, base, base, 2 ** 20, 4, ctypes.byref(q), base, base,
                             ctypes.byref(out), None, base, need.value, None) == OK
    assert lib.stub_attn(1) == 2 ** 24
    lib.ac_layer_destroy(h)
