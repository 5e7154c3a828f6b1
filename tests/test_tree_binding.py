"""CPU: what the Python binding of the tree-speculation calls hands to the library."""

import ctypes

import pytest
import torch

import mqa_decode_attention_gb300 as m
from mqa_decode_attention_gb300 import _abi


def layouts(count):
    return [m.layout_contiguous(*(torch.zeros(2, 2, 64, 128, dtype=torch.bfloat16) for _ in "kv"), 8) for _ in range(count)]


class Recorder:
    """Stands in for the library: the layouts that a keep_path call passes, if they
    are one array as long as the call says (anything else is not looked into)."""

    def __init__(self):
        self.got = None

    def kv_keep_path(self, arg, count, *rest):
        arrays = isinstance(arg, ctypes.Array) and arg._type_ is _abi.KVLayout and len(arg) == count
        self.got = [x.k_cache for x in arg] if arrays else None
        return 0


@pytest.mark.parametrize("form", [list, tuple, m.layout_stack, iter, lambda x: m.layout_stack(x)[0:3]])
def test_keep_path_takes_any_sequence_of_layouts(monkeypatch, form):
    lib = Recorder()
    monkeypatch.setattr(m, "library", lambda: lib)
    lays = layouts(3)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    m.keep_path(form(lays), i32(2), i32(2, 4), i32(2), i32(1), stream=0)
    assert lib.got == [x.k_cache for x in lays]


def test_keep_path_takes_one_layout(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(m, "library", lambda: lib)
    lay = layouts(1)[0]
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    m.keep_path(lay, i32(2), i32(2, 4), i32(2), i32(1), stream=0)
    assert lib.got == [lay.k_cache]


def test_keep_path_refuses_no_layouts_and_other_things():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        m.keep_path([], i32(2), i32(2, 4), i32(2), i32(1), stream=0)
    with pytest.raises(TypeError):
        m.keep_path([1, 2], i32(2), i32(2, 4), i32(2), i32(1), stream=0)


def test_a_list_with_an_invalid_layout_is_refused(built_lib):
    """Through the library itself: the second of a list is looked at, wherever it lies."""
    lays = layouts(2)
    lays[1].head_dim = 96
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(m.MqaError, match="kv_keep_path"):
        m.keep_path(lays, i32(2), i32(2, 4), i32(2), i32(1), stream=0)


def test_layers_that_hold_the_same_rows_are_refused(built_lib):
    """One cache twice in a call would be moved by two blocks at once, a K that is
    its V twice by one. (One pool with a table for each layer is fine: not tried
    here, it would be launched.)"""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    a, b = layouts(2)
    crossed = layouts(1)[0]
    crossed.v_cache = a.k_cache
    same = layouts(1)[0]
    same.v_cache = same.k_cache
    pool = [torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16) for _ in "kv"]
    table = i32(2, 2)
    paged = [m.layout_paged(*pool, table, 8) for _ in "ab"]
    for lays in ([a, b, a], [a, crossed], [same], paged):
        with pytest.raises(m.MqaError, match="invalid argument"):
            m.keep_path(lays, i32(2), i32(2, 4), i32(2), i32(1), stream=0)
