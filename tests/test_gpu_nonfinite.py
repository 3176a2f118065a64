"""A NaN or an infinity in a query, or a NaN in a cached K, makes that row NaN,
however the plan cuts its sequence, and leaves every other row as it is."""

import numpy as np
import pytest
import torch

import gpu_util as gu
import int4_util as iu
from oracle import int4 as oi

pytestmark = pytest.mark.gpu
LENS = [9000, 130, 64, 1, 0, 700]
INT4 = 2


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


def _run(step, q, cache, scale, table, lens):
    step.out.fill_(7.0)
    step.partial_o.fill_(7.0)
    step.partial_lse.fill_(7.0)
    step.plan_step(lens)
    out = step.attend(q, cache, scale, table, lens).clone()
    assert int(step.status.item()) == 0
    return out


def _several(step, b):
    """Items that KV head 0 of sequence b is cut into."""
    return int(step.plan.seg_ptr[8 * b + 1]) - int(step.plan.seg_ptr[8 * b])


@pytest.mark.parametrize("n_ctas", [None, 3])
@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("q_len", [1, 2, 3, 4])
def test_int4_query_that_is_not_finite(q_len, fused, n_ctas):
    from paged_gqa_decode_rope_gb300 import ops
    b = iu.Int4Batch(LENS, 81)
    q = iu.queries((len(LENS), q_len, 64, 128), 82)
    step = ops.DecodeStepEx(len(LENS), INT4, b.max_blocks, q_len=q_len, out_dtype=ops.OUT_FP32, fused=fused,
                            n_ctas=n_ctas)
    args = (b.cache, None, b.block_table, b.seq_lens)
    want = _run(step, q, *args)
    assert _several(step, 0) > 1 or n_ctas
    bad = torch.zeros(want.shape[:3], dtype=torch.bool, device="cuda")
    for s in (0, 1, 2, 5):
        q[s, q_len - 1, 5, 77] = float("nan")
        q[s, q_len - 1, 62, 0] = float("-inf" if s else "inf")
        bad[s, q_len - 1, 5] = bad[s, q_len - 1, 62] = True
    got = _run(step, q, *args)
    assert bool(torch.isnan(got[bad]).all()), "a row that is not finite reads as %s" % got[bad][:, 0].tolist()
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("q_len", [1, 2, 4])
def test_int4_key_that_is_nan(q_len, fused):
    """In every token of one head of a sequence of many items, in the first token
    only of another."""
    from paged_gqa_decode_rope_gb300 import ops
    b = iu.Int4Batch(LENS, 83)
    q = iu.queries((len(LENS), q_len, 64, 128), 84)
    step = ops.DecodeStepEx(len(LENS), INT4, b.max_blocks, q_len=q_len, fused=fused)
    args = (None, b.block_table, b.seq_lens)
    want = _run(step, q, b.cache, *args)
    assert _several(step, 0) > 1
    cache = b.cache.clone()
    nan = torch.tensor([0xC0, 0x7F], dtype=torch.uint8, device="cuda")
    for t in range(LENS[0]):
        blk = int(b.table[0, t // 64])
        for h in (2, 6) if t == 0 else (2,):
            at = oi.scale_byte(0, t % 64, 1)
            cache[blk, h, at:at + 2] = nan
    got = _run(step, q, cache, *args)
    bad = torch.zeros(want.shape[:3], dtype=torch.bool, device="cuda")
    bad[0, :, 16:24] = bad[0, :, 48:56] = True
    assert bool(torch.isnan(got[bad]).all())
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("kv,q_dtype,q_len", [(0, 0, 1), (0, 0, 2), (0, 0, 3), (0, 0, 4), (1, 0, 1), (1, 0, 2),
                                              (1, 0, 3), (1, 0, 4), (1, 1, 1), (1, 1, 2), (1, 1, 4)])
def test_query_that_is_not_finite(kv, q_dtype, q_len, fused):
    """BF16 and E4M3 pages, an E4M3 query among them (which has no infinity)."""
    from paged_gqa_decode_rope_gb300 import ops
    from paged_gqa_decode_rope_gb300.workloads import Workload
    wl = Workload("custom", seed=85, lengths=LENS, kv_dtype=kv, include_new_token=True)
    q = iu.queries((len(LENS), q_len, 64, 128), 86)
    if q_dtype:
        q = q.to(torch.float8_e4m3fn).view(torch.uint8)
    step = ops.DecodeStepEx(len(LENS), kv, wl.max_blocks, q_len=q_len, q_dtype=q_dtype, fused=fused)
    args = (wl.cache, wl.kv_scale, wl.block_table, wl.seq_lens)
    want = _run(step, q, *args)
    assert _several(step, 0) > 1
    bad = torch.zeros(want.shape[:3], dtype=torch.bool, device="cuda")
    for s in (0, 1, 2, 5):
        q[s, q_len - 1, 5, 77] = 0x7F if q_dtype else float("nan")
        q[s, q_len - 1, 62, 0] = 0xFF if q_dtype else float("-inf" if s else "inf")
        bad[s, q_len - 1, 5] = bad[s, q_len - 1, 62] = True
    got = _run(step, q, *args)
    assert bool(torch.isnan(got[bad]).all()), "a row that is not finite reads as %s" % got[bad][:, 0].tolist()
    # (the other rows in bf16: how many items a merge takes at a time depends on
    # which queue makes it, so the last bit of an fp32 sum may differ)
    assert torch.allclose(got[~bad].float(), want[~bad].float(), rtol=2.0 ** -7, atol=0)


@pytest.mark.parametrize("kv,staged", [(0, False), (1, False), (1, True), (2, True)])
def test_prefill_query_that_is_not_finite(kv, staged):
    from paged_gqa_decode_rope_gb300 import ops
    from paged_gqa_decode_rope_gb300.workloads import Workload
    lens, new = [700, 64, 300], [200, 64, 1]
    wl = iu.Int4Batch(lens, 87) if kv == INT4 else \
        Workload("custom", seed=87, lengths=lens, kv_dtype=kv, include_new_token=True)
    q = iu.queries((265, 64, 128), 88)
    qst = torch.tensor([0, 200, 264, 265], dtype=torch.int32, device="cuda")
    pf = ops.PrefillAttention(3, out_dtype=ops.OUT_FP32,
                              staging_pages=ops.PrefillAttention.pages_for(lens) if staged else 0)
    outs = []
    bad = torch.zeros((265, 64), dtype=torch.bool, device="cuda")
    for k in range(2):
        pf.plan(qst)
        outs.append(pf(q, qst, wl.cache, kv, None if kv == INT4 else wl.kv_scale, wl.block_table, wl.seq_lens,
                       torch.full((265, 64, 128), 7.0, device="cuda")))
        assert int(pf.status.item()) == 0
        for i in (0, 130, 199, 230, 264):
            q[i, 5, 77] = float("nan")
            q[i, 62, 0] = float("-inf" if i % 2 else "inf")
            bad[i, 5] = bad[i, 62] = True
    assert bool(torch.isnan(outs[1][bad]).all()), outs[1][bad][:, 0].tolist()
    assert torch.equal(outs[1][~bad], outs[0][~bad])


@pytest.mark.parametrize("out_dtype", [0, 2])
def test_int4_prefill_nan_in_the_cache_reaches_who_sees_it(out_dtype):
    """NaN in K of one new token, in groups of V of others: the tokens before them,
    and other heads, do not see it."""
    from paged_gqa_decode_rope_gb300 import ops
    lens, new = [300, 200, 70], [300, 70, 70]
    b = iu.Int4Batch(lens, 89)
    iu.exact_keys(b)
    clean = b.host.copy()

    def spoil(which, s, t, h, groups):
        for g in groups:
            at = oi.scale_byte(which, t % 64, g)
            b.host[b.table[s, t // 64], h, at:at + 2] = (0xC0, 0x7F)

    spoil(1, 0, 41, 2, [1])           # V of token 41, group 1
    spoil(1, 0, 230, 2, [0, 3])
    spoil(0, 0, 100, 5, [2])          # K of token 100
    spoil(1, 1, 150, 7, range(4))     # V of new token 20
    b.to("cuda")
    q = iu.queries((440, 64, 128), 90)
    qst = torch.tensor([0, 300, 370, 440], dtype=torch.int32, device="cuda")
    pf = ops.PrefillAttention(3, out_dtype=out_dtype, staging_pages=ops.PrefillAttention.pages_for(lens))
    pf.plan(qst)
    out = pf(q, qst, b.cache, INT4, None, b.block_table, b.seq_lens,
             torch.empty(q.shape, dtype=ops._OUT_TORCH[out_dtype], device="cuda"))
    assert int(pf.status.item()) == 0
    gh, qh, dt = iu.host(out), iu.host(q), out.dtype

    def row(s, i, h, nan):
        """Token i of sequence s, a head of KV head h: groups of nan NaN, the others right."""
        at, j = int(qst[s]) + i, 8 * h + i % 8
        K, V = b.rows(s, h, clean)
        want, size = iu.attention(qh[at, j], K, V, lens[s] - new[s] + i + 1)
        bad = np.repeat(np.isin(np.arange(4), list(nan)), 32)
        assert np.all(np.isnan(gh[at, j][bad])), (s, i, h)
        if not bad.all():
            iu.check(gh[at, j][~bad], want[~bad], size[~bad], dt, "seq %d token %d head %d" % (s, i, h))

    for i, nan in ((0, []), (40, []), (41, [1]), (42, [1]), (63, [1]), (64, [1]), (229, [1]), (230, [0, 1, 3]),
                   (299, [0, 1, 3])):
        row(0, i, 2, nan)
        row(0, i, 0, [])
    for i in (0, 70, 99):
        row(0, i, 5, [])
    for i in (100, 101, 128, 299):
        row(0, i, 5, range(4))
    for i in (0, 19):
        row(1, i, 7, [])
    for i in (20, 69):
        row(1, i, 7, range(4))
        row(1, i, 6, [])
    for i in (0, 69):
        row(2, i, 3, [])
