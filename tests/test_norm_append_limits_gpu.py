"""GPU: the normalised append at the ends of its ranges."""

import pytest
import torch

from test_norm_append_gpu import Cache, _check, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m(built_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mqa_decode_attention_gb300 as mod

    mod.library()
    return mod


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [1e-38, 1e-42])
def test_smallest_eps(m, kind, eps):
    """eps down to the smallest numbers, beside rows of zeros and rows whose squares are smaller still: y = x / sqrt(mean
    x^2 + eps) w has a size of its own all the same."""
    B, hq, hkv, d = 6, 4, 4, 128
    c = Cache(m, kind, B, hkv, d, 4, hq)
    x = list(_inputs(kind, B, 1, hq, hkv, d, 21))
    size = torch.tensor([0.0, 1e-25, 1e-21, 1e-19, 1e-16, 1.0]).view(B, 1, 1, 1)
    x[0], x[1] = (x[0].float() * size).to(x[0].dtype), (x[1].float() * size).to(x[1].dtype)
    before = c.snapshot()
    q_rot, err = _run(m, c, 1, x, [1] * B, eps=eps)
    assert err == 0
    _check(c, before, x, [1] * B, q_rot, eps=eps)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_weights_times_largest_values(m, kind):
    """Rows near the end of the range with weights above 1 (x w alone would leave it), and tiny weights."""
    B, hq, hkv, d = 4, 4, 4, 128
    c = Cache(m, kind, B, hkv, d, 4, hq)
    x = list(_inputs(kind, B, 1, hq, hkv, d, 22))
    size = torch.tensor([1e37, 5e37, 2e19, 1e30]).view(B, 1, 1, 1)
    x[0], x[1] = (x[0].float() * size).to(x[0].dtype), (x[1].float() * size).to(x[1].dtype)
    x[4] = (x[4].float() * 64).to(x[4].dtype)
    before = c.snapshot()
    q_rot, err = _run(m, c, 1, x, [1] * B)
    assert err == 0
    _check(c, before, x, [1] * B, q_rot)
