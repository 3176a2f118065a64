"""Block tables and slot maps built on the device against a plain simulation,
and a serving run over the 4-bit cache that uses them: prompts, decode steps,
rejected drafts, finished requests."""

import numpy as np
import pytest
import torch

import gpu_util as gu
import int4_util as iu

pytestmark = pytest.mark.gpu
BAD_BLOCK, BAD_SEQ_LEN, PLAN_OVERFLOW, OUT_OF_BLOCKS = 1, 4, 16, 128


@pytest.fixture(autouse=True)
def _gpu():
    gu.require_gpu()


class Plain:
    """The same bookkeeping on the host, one request and one token at a time."""

    def __init__(self, batch, max_blocks, num_blocks, max_tokens):
        self.table = np.full((batch, max_blocks), -1, dtype=np.int64)
        self.free = list(range(num_blocks - 1, -1, -1))
        self.num_blocks, self.max_tokens, self.status = num_blocks, max_tokens, 0

    def step(self, hist, new):
        B, mb = self.table.shape
        lens, start = np.zeros(B, dtype=np.int64), [0]
        pos, slot = np.zeros(self.max_tokens, dtype=np.int64), np.full(self.max_tokens, -1, dtype=np.int64)
        stop = False
        for b in range(B):
            h, n = int(hist[b]), int(new[b])
            at = start[-1]
            start.append(at + max(n, 0))
            if h < 0 or n < 0 or h + n > mb * 64:
                self.status |= BAD_SEQ_LEN
                continue
            if at + n > self.max_tokens:
                self.status |= PLAN_OVERFLOW
                continue
            want = -(-(h + n) // 64) - -(-h // 64)
            if want and (stop or want > len(self.free)):
                stop = True
                self.status |= OUT_OF_BLOCKS
                continue
            for j in range(-(-h // 64), -(-(h + n) // 64)):
                self.table[b, j] = self.free.pop()
            lens[b] = h + n
            for i in range(n):
                p = h + i
                blk = self.table[b, p // 64]
                pos[at + i] = p
                if 0 <= blk < self.num_blocks:
                    slot[at + i] = blk * 64 + p % 64
                else:
                    self.status |= BAD_BLOCK
        return lens, np.array(start), pos, slot

    def release(self, lens, keep):
        back = []
        for b in range(len(lens)):
            back += [self.table[b, j] for j in range(-(-int(keep[b]) // 64), -(-int(lens[b]) // 64))]
        self.free += back[::-1]


def _dev(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _same(t, p, want, status=None):
    lens, start, pos, slot = want
    assert np.array_equal(t.seq_lens.cpu().numpy(), lens)
    assert np.array_equal(t.query_start.cpu().numpy(), start)
    assert np.array_equal(t.positions.cpu().numpy(), pos)
    assert np.array_equal(t.slot_mapping.cpu().numpy(), slot)
    assert np.array_equal(t.block_table.cpu().numpy(), p.table)
    n, ticket = t.pool.tolist()
    assert n == len(p.free) and ticket == 0
    assert t.free_blocks.cpu().numpy()[:n].tolist() == p.free
    assert int(t.status.item()) == (p.status if status is None else status)


def _pair(batch, max_blocks, num_blocks, max_tokens):
    from paged_gqa_decode_rope_gb300 import ops
    return (ops.BlockTables(batch, max_blocks, num_blocks, max_tokens),
            Plain(batch, max_blocks, num_blocks, max_tokens))


@pytest.mark.parametrize("batch,most,max_tokens", [(1, 1, 1), (1, 5000, 5003), (5, 200, 900), (37, 64, 4000),
                                                   (300, 130, 40000), (8192, 3, 20001)])
def test_steps_match_the_plain_form(batch, most, max_tokens):
    r = np.random.default_rng(batch)
    t, p = _pair(batch, 90, batch * 8 + 90, max_tokens)
    hist = np.zeros(batch, dtype=np.int64)
    for k in range(5):
        room = np.minimum(90 * 64 - hist, max(1, max_tokens // batch))
        new = np.minimum(r.integers(0, most + 1, batch), room)
        if k == 2:
            new[r.random(batch) < 0.5] = 0
        want = p.step(hist, new)
        t.step(_dev(hist), _dev(new))
        _same(t, p, want)
        lens = np.where(want[0] > 0, want[0], hist)
        # some requests finish, some give back part of what they took
        keep = np.where(r.random(batch) < 0.2, 0, np.where(r.random(batch) < 0.3, lens - new // 2, lens))
        keep = np.clip(keep, 0, lens)
        p.release(lens, keep)
        t.release(_dev(lens), _dev(keep))
        _same(t, p, want)
        hist = keep


def test_release_of_a_step_restores_the_pool():
    t, p = _pair(50, 20, 900, 30000)   # room for every token: 50 x 599, then 50 x 129
    r = np.random.default_rng(2)
    hist = r.integers(0, 600, 50)
    t.step(_dev(np.zeros(50)), _dev(hist))
    before, free = t.pool.clone(), t.free_blocks.clone()
    t.step(_dev(hist), _dev(r.integers(0, 130, 50)))
    assert int(t.status.item()) == 0
    assert not torch.equal(t.pool, before)
    t.release(t.seq_lens, _dev(hist))
    assert torch.equal(t.pool, before)
    n = int(before[0])
    assert torch.equal(t.free_blocks[:n], free[:n])


def test_a_dry_pool_serves_in_order():
    t, p = _pair(6, 10, 7, 2000)
    hist = np.array([0, 0, 0, 0, 0, 0])
    new = np.array([130, 64, 200, 1, 0, 3])       # 3 + 1 + 4 (too many) + 1, 0, 1
    want = p.step(hist, new)
    t.step(_dev(hist), _dev(new))
    assert p.status == OUT_OF_BLOCKS and want[0].tolist() == [130, 64, 0, 0, 0, 0]
    _same(t, p, want)


def test_bad_lengths_and_full_step():
    t, p = _pair(8, 4, 40, 300)
    hist = np.array([-1, 0, 250, 10, 0, 256, 0, 1])
    new = np.array([5, -3, 7, 20, 250, 0, 100, 2])   # bad, bad, too long, ok, ok, ok, past 300, past 300
    p.table[2, :4] = [36, 37, 38, 39]
    p.table[3, 0], p.table[5] = 35, [31, 32, 33, 34]
    p.table[7, 0] = 30
    t.block_table.copy_(_dev(p.table))
    want = p.step(hist, new)
    assert want[0].tolist() == [0, 0, 0, 30, 250, 256, 0, 0]
    assert p.status == BAD_SEQ_LEN | PLAN_OVERFLOW
    t.step(_dev(hist), _dev(new))
    _same(t, p, want)


def test_bad_block_ids():
    t, p = _pair(3, 4, 8, 64)
    p.table[0, 0], p.table[1, 0] = 8, -1
    t.block_table.copy_(_dev(p.table))
    hist, new = np.array([5, 5, 0]), np.array([3, 2, 4])
    p.free[-1] = 99
    t.free_blocks.copy_(_dev(p.free))
    want = p.step(hist, new)
    t.step(_dev(hist), _dev(new))
    assert p.status == BAD_BLOCK and np.all(want[3] == -1)
    _same(t, p, want)


def test_release_refuses_what_does_not_fit():
    t, _ = _pair(3, 4, 8, 64)
    t.block_table.fill_(3)
    t.release(_dev([64, 0, 0]), _dev([0, 0, 0]))          # the pool is full already
    assert int(t.status.item()) == PLAN_OVERFLOW and t.pool.tolist() == [8, 0]
    t.status.zero_()
    t.pool[0] = 0
    t.release(_dev([-1, 300, 64]), _dev([0, 0, 65]))      # negative, too long, keep > len
    assert int(t.status.item()) == BAD_SEQ_LEN and t.pool.tolist() == [0, 0]
    t.status.zero_()
    t.block_table[2, 1] = 8
    t.release(_dev([0, 0, 128]), _dev([0, 0, 10]))
    assert int(t.status.item()) == BAD_BLOCK and t.pool.tolist() == [1, 0]


def test_captured_steps_replay():
    """A captured build and release, replayed on new lengths; the padded tail keeps slot -1."""
    t, p = _pair(16, 40, 400, 1000)
    hist, new = _dev(np.zeros(16)), _dev(np.zeros(16))
    t.step(hist, new)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.step(hist, new)
    r = np.random.default_rng(3)
    h = np.zeros(16, dtype=np.int64)
    for _ in range(4):
        n = r.integers(0, 60, 16)
        hist.copy_(_dev(h))
        new.copy_(_dev(n))
        g.replay()
        want = p.step(h, n)
        _same(t, p, want)
        h = want[0]


def test_serving_run_over_the_4bit_cache():
    """Prompts admitted together, then decode steps with drafts, one of them
    rejected, and a request that ends: every attention output against the exact
    attention over what the cache holds."""
    from oracle import int4 as oi
    from paged_gqa_decode_rope_gb300 import ops
    B, mb, KV = 5, 6, 2
    t = ops.BlockTables(B, mb, 40, 512)
    cache = ops.int4_cache(40)
    cos_sin = ops.rope_cos_sin_cache(mb * 64)
    w = (1 + 0.1 * torch.randn(128, device="cuda")).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hist = np.zeros(B, dtype=np.int64)

    def tokens(seed):
        q, k, v = (iu.queries((512, n, 128), seed + n) for n in (64, 8, 9))
        v = v[:, :8].contiguous()
        q_out = torch.zeros_like(q)
        ops.rope_norm_kvwrite(q, k, v, t.positions, cos_sin, w, w, cache, KV, t.slot_mapping, None, q_out, status)
        return q_out

    def check(out, q_out, new):
        host, table, starts = cache.cpu().numpy(), t.block_table.cpu().numpy(), t.query_start.tolist()
        for b in range(B):
            L = int(hist[b] + new[b])
            K, V = (x[:L] for x in oi.read_rows(host, table[b, :-(-L // 64)], 3))
            for i in sorted({0, int(new[b]) // 2, int(new[b]) - 1}) if new[b] else []:
                row = starts[b] + i
                want, size = iu.attention(iu.host(q_out[row, 25]), K, V, int(hist[b]) + i + 1)
                iu.check(iu.host(out[row, 25]), want, size, torch.bfloat16, "seq %d token %d" % (b, i))

    # prompts
    new = np.array([70, 1, 64, 0, 130])
    t.step(_dev(hist), _dev(new))
    q_out = tokens(100)
    pf = ops.PrefillAttention(B, staging_pages=30)
    pf.plan(t.query_start)
    out = torch.zeros((512, 64, 128), dtype=torch.bfloat16, device="cuda")
    pf(q_out, t.query_start, cache, KV, None, t.block_table, t.seq_lens, out)
    check(out, q_out, new)
    hist = hist + new
    # two steps of two draft tokens; the second draft of every other request is rejected
    step = ops.DecodeStepMT(B, 2, KV, mb)
    for k in range(2):
        new = np.full(B, 2)
        t.step(_dev(hist), _dev(new))
        q_out = tokens(200 + k)
        step.plan_step(t.seq_lens)
        out = step.attend(q_out[:2 * B].view(B, 2, 64, 128), cache, None, t.block_table, t.seq_lens)
        check(out.view(2 * B, 64, 128), q_out, new)
        keep = hist + 2 - (np.arange(B) % 2)
        t.release(t.seq_lens, _dev(keep))
        hist = keep
    # request 2 ends, another takes its row
    lens = hist.copy()
    hist = np.where(np.arange(B) == 2, 0, hist)
    t.release(_dev(lens), _dev(hist))
    one = ops.DecodeStep(B, KV, mb)
    new = np.ones(B, dtype=np.int64)
    t.step(_dev(hist), _dev(new))
    q_out = tokens(300)
    one.plan_step(t.seq_lens)
    out = one.attend(q_out[:B].contiguous(), cache, None, t.block_table, t.seq_lens)
    check(out, q_out, new)
    used = sum(-(-int(x) // 64) for x in hist + new)
    assert t.pool.tolist() == [40 - used, 0]
    for s in (status, t.status, pf.status, step.status, one.status):
        assert int(s.item()) == 0


def test_calls_without_entries():
    """No sequences, no tokens, no slots: nothing to do is no error."""
    from paged_gqa_decode_rope_gb300 import ops
    t, p = _pair(0, 4, 9, 5)                              # no sequences, all rows padding
    want = p.step([], [])
    t.step(_dev([]), _dev([]))
    _same(t, p, want)
    t.release(_dev([]), _dev([]))
    _same(t, p, want)
    t, p = _pair(3, 4, 9, 0)                              # no room for tokens
    want = p.step([5, 0, 64], [0, 0, 0])
    t.step(_dev([5, 0, 64]), _dev([0, 0, 0]))
    _same(t, p, want)
    for kv, cache in ((0, torch.zeros((2, 2, 8, 64, 128), dtype=torch.bfloat16, device="cuda")), (2, ops.int4_cache(2))):
        k, v = (torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ops.kv_gather(cache, kv, None, torch.empty(0, dtype=torch.int64, device="cuda"), k, v, t.status)
    assert int(t.status.item()) == 0
