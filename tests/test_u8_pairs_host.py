"""CPU: a uint8 layout takes the pairs of uint8 rows only. Others, such as the bf16 pairs of a 4-bit cache whose
cache_dtype was left out, hold fewer bytes than the kernels read and write."""

import warnings

import pytest
import torch

import mqa_decode_attention_gb300 as m
from mqa_decode_attention_gb300 import _abi

B, HQ, HKV, ROWS, D = 2, 4, 2, 16, 64


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib):
    return _abi.load()


def _pairs(dtype=torch.float32, rows=ROWS):
    return torch.zeros(B, HKV, rows, 2, dtype=dtype)


def _codes():
    return torch.zeros(B, HKV, ROWS, D, dtype=torch.uint8)


def _layout(paged, ksz, vsz):
    if paged:
        return m.layout_paged(_codes(), _codes(), torch.zeros(B, 3, dtype=torch.int32), HQ, 0, ksz, vsz)
    return m.layout_contiguous(_codes(), _codes(), HQ, 0, ksz, vsz)


UNFIT = {
    "a 4-bit cache's": lambda: _pairs(torch.bfloat16),
    "float64": lambda: _pairs(torch.float64),
    "too few": lambda: _pairs(rows=ROWS - 2),
    "not dense": lambda: torch.zeros(B, HKV, ROWS, 4)[..., ::2],
}


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("name", list(UNFIT))
def test_unfit_pairs_are_refused(name, which, paged):
    """The layout has no pairs, with a warning, and every call that takes it is an invalid argument before any launch."""
    pairs = [_pairs(), _pairs()]
    pairs[which] = UNFIT[name]()
    with pytest.warns(UserWarning, match="float32"):
        lay = _layout(paged, *pairs)
    bf, i32 = torch.bfloat16, torch.int32
    q, kv = torch.zeros(B, 1, HQ, D, dtype=bf), torch.zeros(B, 1, HKV, D, dtype=bf)
    pos, err, rot, out = torch.zeros(B, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(B, 1, HQ, D), torch.zeros(B, 1, HQ, D)
    rows = [torch.zeros(B, HKV, 4, D) for _ in "kv"]
    bufs = m.DecodeBuffers(rot, out, torch.zeros(B, 1, HQ), None, err)
    calls = [
        lambda: m.kv_append_rope(lay, q, kv, kv, pos, 1e4, rot, err, stream=0),
        lambda: m.kv_append_rope_multi(lay, 1, q, kv, kv, pos, 1e4, rot, err, stream=0),
        lambda: m.kv_append_norm_rope(lay, 1, q, kv, kv, pos, 1e4, rot, err, stream=0),
        lambda: m.gqa_decode_attention(lay, rot, pos, 8, 0.1, 1, out, err=err, stream=0),
        lambda: m.gqa_decode_attention_multi(lay, 1, rot, pos, 8, 0.1, 1, out, err=err, stream=0),
        lambda: m.decode_step(lay, q, kv, kv, pos, pos, 8, bufs, num_splits=1, stream=0),
        lambda: m.kv_read_rows(lay, None, None, *rows, err, stream=0),
    ]
    for call in calls:
        with pytest.raises(m.MqaError) as e:
            call()
        assert e.value.status == _abi.MQA_ERR_INVALID_ARG


def test_fit_pairs_are_taken():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for paged in (False, True):
            for pairs in (_pairs(), _pairs().view(B, HKV, 2 * ROWS), _pairs(rows=ROWS + 4)):
                lay = _layout(paged, pairs, pairs)
                assert lay.cache_dtype == m.MQA_U8 and lay.k_scale_zero == lay.v_scale_zero == pairs.data_ptr()
            _layout(paged, None, None)  # (as before: the calls refuse it)
