"""GPU: steps over a 4-bit cache whose attention has nothing to do, waits of its wider kernels that run out, large caches."""

import math

import pytest
import torch

from u4_cases import U4Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m(built_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mqa_decode_attention_gb300 as mod

    mod.library()
    return mod


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("page", [0, 16])
def test_step_of_lengths_out_of_range(m, page, splits):
    """Every length is out of range, so that all blocks of the attention leave at once: what follows on the stream still
    finds the rows that the step appended."""
    B, hq, hkv, d, n = 48, 8, 8, 128, 32
    c = U4Case(hq, hkv, d, [256] * B, n, page, seed=3, garbage=False)
    g = torch.Generator().manual_seed(5)
    new = [torch.randn(B, n, h, d, generator=g).to(torch.bfloat16).to(DEV) for h in (hq, hkv, hkv)]
    lay = c.layout(m)
    bufs = m.DecodeBuffers.allocate(lay, 256, num_splits=splits, n_new=n)
    want = {}
    pos, rot, err = _i32([11] * B), torch.empty(B, n, hq, d, device=DEV), _i32([0])
    m.kv_append_rope_multi(lay, n, *new, pos, 10000.0, rot, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    want = {x: c.dev[x].clone() for x in ("k", "v", "ksm", "vsm")}
    lens = _i32([0, 257, -3, 31] * (B // 4))
    for _ in range(5):
        for x in want:
            c.dev[x].zero_()
        bufs.err.zero_()
        m.decode_step_multi(lay, n, *new, pos, lens, 256, bufs, scale=1 / math.sqrt(d), num_splits=splits)
        found = {x: c.dev[x].clone() for x in want}  # on the same stream, right behind the step
        torch.cuda.synchronize()
        assert int(bufs.err) == m.MQA_DEVERR_SEQ_LEN
        for x in want:
            for b in range(0, B, 7):
                for t in range(11, 11 + n):
                    at = c.slot(b, t)
                    assert torch.equal(found[x][at].view(torch.uint8), want[x][at].view(torch.uint8)), (x, b, t)


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("group,splits", [(12, 1), (12, 2), (32, 1), (32, 2)])
def test_timeout_of_wider_kernels(m, group, splits, page):
    """The waits of the 16-row and 32-row kernels and of paged tiles with a limit of 1 ns: the call comes back, says so, and
    the next one gives what the call before gave."""
    B, hkv, d, L = 24, 4, 128, 6000
    g = torch.Generator(DEV).manual_seed(7)
    shape = (B * -(-L // 16), hkv, 16) if page else (B, hkv, L)
    codes = [torch.randint(0, 256, (*shape, d // 2), generator=g, dtype=torch.uint8, device=DEV) for _ in "kv"]
    pairs = [torch.rand(*shape, 2, generator=g, device=DEV).to(torch.bfloat16) for _ in "kv"]
    if page:
        table = torch.randperm(shape[0], generator=g, device=DEV).int().view(B, -1)
        lay = m.layout_paged(codes[0], codes[1], table, hkv * group, 0, pairs[0], pairs[1], cache_dtype=m.MQA_U4)
    else:
        lay = m.layout_contiguous(codes[0], codes[1], hkv * group, 0, pairs[0], pairs[1], cache_dtype=m.MQA_U4)
    q, lens = torch.randn(B, hkv * group, d, generator=g, device=DEV), _i32([L] * (B - 2) + [L - 77, 130])
    bufs = m.DecodeBuffers.allocate(lay, L, num_splits=splits)

    def call():
        bufs.err.zero_()
        m.gqa_decode_attention(lay, q, lens, L, 0.09, splits, bufs.out, bufs.lse, bufs.workspace, err=bufs.err)
        torch.cuda.synchronize()
        return int(bufs.err), bufs.out.clone()

    err, before = call()
    assert err == 0 and torch.isfinite(before).all()
    lay.wait_limit_ns = 1
    for _ in range(5):
        err, out = call()
        # (a wait that finds its tile at the first look does not run out: 32 rows take longer over a tile than its load)
        assert err == m.MQA_DEVERR_TIMEOUT or (err == 0 and torch.equal(before, out))
    lay.wait_limit_ns = 0
    err, after = call()
    assert err == 0 and torch.equal(before, after)


@pytest.mark.parametrize("page", [0, 16])
def test_offsets_past_32_bits(m, page):
    """The last of 68 sequences of 2^20 rows: its codes lie past 2^32 bytes. Appended, attended to and read back as in a
    small cache, bit for bit."""
    B, hq, hkv, d, rows, n = 68, 4, 1, 128, 1 << 20, 3
    small = U4Case(hq, hkv, d, [300], n, seed=9, garbage=False)
    g = torch.Generator().manual_seed(2)
    new = [torch.randn(1, n, h, d, generator=g).to(torch.bfloat16).to(DEV) for h in (hq, hkv, hkv)]
    shape = (B * rows // 16, hkv, 16) if page else (B, hkv, rows)
    codes = [torch.zeros(*shape, d // 2, dtype=torch.uint8, device=DEV) for _ in "kv"]
    pairs = [torch.zeros(*shape, 2, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    if page:  # 19 pages of the sequence, the last of the pool, from the last one down
        pages = shape[0] - 1 - torch.arange(19)
        table = pages.int().view(1, 19).to(DEV)
        for t in range(300):
            for x, y in zip(codes + pairs, (small.k, small.v, small.ksm, small.vsm)):
                x[int(pages[t // 16]), :, t % 16] = y[0, :, t].to(DEV)
        lay = m.layout_paged(codes[0], codes[1], table, hq, 0, pairs[0], pairs[1], cache_dtype=m.MQA_U4)
        first, batch = 0, 1
    else:
        for x, y in zip(codes + pairs, (small.k, small.v, small.ksm, small.vsm)):
            x[-1, :, : y.shape[2]] = y[0].to(DEV)
        lay = m.layout_contiguous(codes[0], codes[1], hq, 0, pairs[0], pairs[1], cache_dtype=m.MQA_U4)
        first, batch = B - 1, B
    ref = small.layout(m)
    outs = []
    for layout, at, size in ((ref, 0, 1), (lay, first, batch)):
        x = [torch.zeros(size, *t.shape[1:], dtype=t.dtype, device=DEV) for t in new]
        for a, b in zip(x, new):
            a[at] = b[0]
        pos = torch.zeros(size, dtype=torch.int32, device=DEV)
        pos[at] = 297
        bufs = m.DecodeBuffers.allocate(layout, 300, num_splits=2, n_new=n)
        m.decode_step_multi(layout, n, *x, pos, pos + n, 300, bufs, num_splits=2)
        w = torch.full((d,), 1.25, dtype=torch.bfloat16, device=DEV)
        rows_out = [torch.zeros(size, hkv, 300, d, device=DEV) for _ in "kv"]
        m.kv_read_rows(layout, None, pos + n, *rows_out, bufs.err)
        step = [bufs.out[at].clone()] + [r[at].clone() for r in rows_out]
        m.kv_append_norm_rope(layout, n, *x, pos, 1e4, bufs.q_rot, bufs.err, q_weight=w, k_weight=w)
        m.kv_read_rows(layout, None, pos + n, *rows_out, bufs.err)
        torch.cuda.synchronize()
        assert int(bufs.err) == 0
        outs.append(step + [r[at].clone() for r in rows_out])
    # (the runs of tiles differ with the number of units: the output within its bf16 rounding and the sums' order)
    assert torch.all((outs[0][0].float() - outs[1][0].float()).abs() <= 16 * (2.0 ** -11 + 2.0 ** -16) + 1.01 * 2.0 ** -7 * outs[0][0].float().abs())
    for a, b in zip(outs[0][1:], outs[1][1:]):
        assert torch.equal(a, b)
