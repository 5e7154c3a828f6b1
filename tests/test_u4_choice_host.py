"""CPU: which contiguous batches over a 4-bit cache get one block for each unit when the library chooses."""

import ctypes

import pytest

from mqa_decode_attention_gb300 import _abi

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib(built_lib):
    return _abi.load()


def _choice(lib, most, n=1, window=0, batch=64, h_q=32, head_dim=128):
    lay = _abi.KVLayout(cache_dtype=_abi.MQA_U4, batch=batch, h_q=h_q, h_kv=8, head_dim=head_dim, paged=0, k_cache=FAKE, v_cache=FAKE,
                        capacity=1 << 20, page_size=0, num_pages=0, max_pages_per_seq=0, window=window, block_table=None,
                        k_scale_zero=FAKE, v_scale_zero=FAKE)
    choice = lib.mqa_choose_splits_multi(ctypes.byref(lay), n, most, 0)
    size = lib.mqa_workspace_size_multi(ctypes.byref(lay), n, most, 0, 0)
    assert (size > 0) == (choice > 1)
    return choice


def test_many_units_of_bounded_length(lib):
    """The lengths are only bounded: one of them may be the bound and the others short, and a block that takes a whole unit
    then works alone. Up to 128 tiles that costs less than equal parts gain; past them tiles are shared."""
    for kw in (dict(), dict(n=4), dict(n=8), dict(head_dim=64)):
        assert _choice(lib, 8192, **kw) == 1, kw
        assert _choice(lib, 8193, **kw) == 2, kw
        assert _choice(lib, 131072, **kw) == 2, kw
    assert _choice(lib, 131072, window=4096) == 1  # what a window leaves counts
    assert _choice(lib, 131072, window=16384) == 2


def test_choices_do_not_grow_a_workspace(lib):
    """A workspace that was made for a bound serves every smaller one."""
    for kw in (dict(), dict(n=8), dict(batch=4), dict(batch=16), dict(h_q=64, n=4)):
        picks = [_choice(lib, most, **kw) for most in (32, 300, 1024, 1025, 4096, 8192, 8193, 60000, 1 << 20)]
        assert picks == sorted(picks), (kw, picks)
